// ss_ffn.cuh -- what the kernels of the gated feed-forward block share: the
// activations with their slopes, the problems as the launchers take them, and
// the choice between the two families of kernels.
//
// The block's seven products are all of the form Out[n, m] = sum_k B[n, k] A[m, k]
// with operands that TMA brings to shared memory as they lie (K-major, or
// MN-major through the MMA's operand descriptor), so nothing is transposed:
//   gate/up  G, U [T, F]  X [T, D] (K-major)      Wg, Wu [F, D] (K-major)
//   down     Z  [T, D]    A [T, F] (K-major)      Wd [D, F] (K-major)
//   dA       dA [T, F]    dZ [T, D] (K-major)     Wd [D, F] (MN-major)
//   dX       dX [T, D]    dG, dU [T, F] (K-major) Wg, Wu [F, D] (MN-major)
//   dW       dWg [F, D]   dG [T, F] (MN-major)    X [T, D] (MN-major); dWu and
//            dWd (dZ, A) likewise
// Two families run them: ss_ffn_pair.cu on CTA pairs with 256 x 256 tiles, and
// ss_ffn_split.cu with smaller tiles and K split over a thread-block cluster,
// for problems whose tiles would leave most SMs idle.
#pragma once

#include <type_traits>

#include "ss_dropout.cuh"
#include "ss_ffn_plan.h"
#include "ss_internal.h"
#include "ss_ptx.cuh"
#include "ss_shared.h"

namespace ss {

// ------------------------------------------------------------- activations

// sigmoid(x) = 1 / (1 + 2^(-x log2 e)): exactly 0 and 1 at the ends
__device__ __forceinline__ float sigmoid_fast(float x) {
  return rcp_approx(1.f + ex2_approx(-1.4426950408889634f * x));
}

// The normal distribution's Phi(g), from e = exp(-g^2 / 2): Phi(-|g|) / e is
// smooth, and t P(t) in t = 1 / (1 + 0.3 |g|) with the coefficients below, which
// least squares reweighted towards the largest error (Lawson) gave for |g| up to
// 14, is off by 1.7e-7 of it. So the left tail, which (1 + erf) / 2 cancels away
// (0.2% off at -4), keeps its digits, and one exponential serves Phi and density.
__device__ __forceinline__ float normal_cdf(float g, float e) {
  const float t = rcp_approx(fmaf(0.3f, fabsf(g), 1.f));
  float p = fmaf(t, 0.035674762f, -0.157203019f);
  p = fmaf(t, p, 0.206353411f);
  p = fmaf(t, p, -0.0536835454f);
  p = fmaf(t, p, 0.128561571f);
  p = fmaf(t, p, 0.0999135077f);
  p = fmaf(t, p, 0.120753951f);
  p = fmaf(t, p, 0.119629301f);
  const float q = e * t * p;
  return g < 0.f ? q : 1.f - q;
}

// a = act(g), and (SLOPE) d = act'(g)
template <int ACT, bool SLOPE>
__device__ __forceinline__ void act_eval(float g, float& a, float& d) {
  if constexpr (ACT == SS_ACT_SILU) {
    const float s = sigmoid_fast(g);
    a = g * s;
    if (SLOPE) d = fmaf(a, 1.f - s, s);
  } else if constexpr (ACT == SS_ACT_GELU) {
    const float e = ex2_approx(-0.72134752044448170f * g * g);  // exp(-g^2 / 2)
    const float cdf = normal_cdf(g, e);
    a = g * cdf;
    if (SLOPE) d = fmaf(g * 0.39894228040143268f, e, cdf);  // the density is e / sqrt(2 pi)
  } else if constexpr (ACT == SS_ACT_GELU_TANH) {
    // (1 + tanh v) / 2 = sigmoid(2 v), 2 v = c (g + 0.044715 g^3), c = 2 sqrt(2 / pi)
    constexpr float c = 1.5957691216057308f;
    const float g2 = g * g;
    const float s = sigmoid_fast(c * g * fmaf(0.044715f, g2, 1.f));
    a = g * s;
    // where g^2 is past 10^4, s is 0 or 1 and the factor (1 - s) a is 0: the
    // bound keeps 0 * infinity out
    if (SLOPE) d = fmaf(a * (1.f - s), c * fmaf(0.134145f, fminf(g2, 1e4f), 1.f), s);
  } else {
    a = g < 0.f ? 0.f : g;  // a NaN stays
    if (SLOPE) d = g > 0.f ? 1.f : 0.f;
  }
}

// fn.template operator()<ACT>() for the activation `act`
template <class F>
__device__ __forceinline__ void dispatch_act(int act, F&& fn) {
  switch (act) {  // uniform
    case SS_ACT_SILU: fn(std::integral_constant<int, SS_ACT_SILU>{}); break;
    case SS_ACT_GELU: fn(std::integral_constant<int, SS_ACT_GELU>{}); break;
    case SS_ACT_GELU_TANH: fn(std::integral_constant<int, SS_ACT_GELU_TANH>{}); break;
    default: fn(std::integral_constant<int, SS_ACT_RELU>{}); break;
  }
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Barrier `id` of `nthreads` threads in whole warps, after code in which the lanes
// of a warp part (one lane's arrival or copy): it wants the warp whole, which the
// compiler does not see in inline assembly.
__device__ __forceinline__ void group_sync(int id, int nthreads) {
  __syncwarp();
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// 32 bytes per lane, one whole sector (32-byte aligned addresses).
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void ld_global_v8(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// the same with a second constant: whether low bits of G and U (below) are there
template <class F>
__device__ __forceinline__ void dispatch_act_low(int act, bool low, F&& fn) {
  dispatch_act(act, [&](auto a) {
    if (low) fn(a, std::true_type{});  // uniform
    else fn(a, std::false_type{});
  });
}

// ------------------------------------------ four more bits of G and of U each
//
// The backward takes its factors from G and U, which the forward keeps in bf16;
// their rounding would be half of the backward's own error. One byte per element
// holds the next four bits of each, G's in the low and U's in the high half: 8
// plus the distance of the fp32 value from its rounded one in 16ths of a bf16
// step. (Bit patterns of floats of one sign are ordered like their magnitudes, so
// integer differences of them are distances in steps.)
//
// Measured at T 8192, D 2048, F 5504: forward and backward together are off by
// 2.4e-3 of the gradients' norm, without these bits by 3.1e-3. They cost a byte to
// the six that are kept per element: the forward of T 16384, D 768, F 2048 takes
// 134 us instead of 128, its backward 253 instead of 245 (T 65536: 490 for 460 and
// 957 for 930).

// That distance in 65536ths of a step (2^15 at most either way) plus 8 and a half
// 16ths: bits 12 to 15 are the half byte, rounded to nearest. 15 is the largest.
__device__ __forceinline__ uint32_t low_bits(float x, uint32_t hi) {
  return static_cast<uint32_t>(
      __viaddmin_s32(static_cast<int>(__float_as_uint(x) - hi), 0x8800, 0xffff));
}
// byte 1 of each of four words
__device__ __forceinline__ uint32_t second_bytes(const uint32_t (&d)[4]) {
  return __byte_perm(__byte_perm(d[0], d[1], 0x0051), __byte_perm(d[2], d[3], 0x0051), 0x5410);
}
// the low bits of four elements, from their fp32 values and packed bf16 pairs
__device__ __forceinline__ uint32_t low_bits4(const float (&g)[4], const float (&u)[4],
                                              uint32_t g01, uint32_t g23, uint32_t u01,
                                              uint32_t u23) {
  const uint32_t dg[4] = {low_bits(g[0], g01 << 16), low_bits(g[1], g01 & 0xffff0000u),
                          low_bits(g[2], g23 << 16), low_bits(g[3], g23 & 0xffff0000u)};
  const uint32_t du[4] = {low_bits(u[0], u01 << 16), low_bits(u[1], u01 & 0xffff0000u),
                          low_bits(u[2], u23 << 16), low_bits(u[3], u23 & 0xffff0000u)};
  return (second_bytes(du) & 0xf0f0f0f0u) | ((second_bytes(dg) >> 4) & 0x0f0f0f0fu);
}
// The half bytes of four elements of G or of U, each in the upper half of its byte.
__device__ __forceinline__ uint32_t halves_g(uint32_t low) { return (low << 4) & 0xf0f0f0f0u; }
__device__ __forceinline__ uint32_t halves_u(uint32_t low) { return low & 0xf0f0f0f0u; }
// Element k (0 to 3) of four: the bf16 (the pair's second where k is odd) above its
// half byte twice, less 8 of them; the second is a 256th of the first and saves
// clearing what is below it.
__device__ __forceinline__ float refine(uint32_t pair, uint32_t halves, int k) {
  const uint32_t sel = (k & 1 ? 0x3200u : 0x1000u) + static_cast<uint32_t>(4 + k) * 0x11u;
  return __int_as_float(static_cast<int>(__byte_perm(pair, halves, sel)) - 0x8080);
}

// ---------------------------------------------------------------- problems

struct FfnForward {
  const uint16_t *X, *Wg, *Wu, *Wd, *residual;
  int T, D, F, act;
  DropArgs drop;
  uint16_t *Y, *G, *U, *A;  // G, U null: not kept
  int ldo;                  // elements between the rows of G, U and A
  uint8_t* R;               // nullable: low bits of G and U
  int ldr;                  // bytes between the rows of R
  int* status;
  int num_sms;
};

struct FfnBackward {
  const uint16_t *dZ, *X, *Wg, *Wu, *Wd, *G, *U, *A;  // dZ: dY with dropped elements zeroed
  int T, D, F, act;
  float scale;  // 1 / (1 - p): dZ above times this is the gradient of Z
  int dw_fp32, accumulate;
  const uint8_t* R;  // nullable: low bits of G and U
  int ldr;
  uint16_t *dX, *dG, *dU;
  int ldg;  // elements between the rows of dG and dU
  void *dWg, *dWu, *dWd;
  int* status;
  int num_sms;
};

// ---------------------------------------------------------- tiles and maps

inline int tiles_of(int64_t n, int tile) { return static_cast<int>(cdiv(n, tile)); }

// K-major operand [rows, k]: boxes of box_rows rows x 64 of k. MN-major operand
// [k, cols]: boxes of 64 columns x 64 of k. ld: elements between rows.
inline bool map_kmajor(CUtensorMap* m, const uint16_t* p, int64_t rows, int64_t k, int64_t ld,
                       int box_rows = 128) {
  return make_bf16_map(m, p, k, rows, ld * 2, 64, box_rows);
}
inline bool map_mnmajor(CUtensorMap* m, const uint16_t* p, int64_t k, int64_t cols, int64_t ld) {
  return make_bf16_map(m, p, cols, k, ld * 2, 64, 64);
}

// ------------------------------------------------------------- the kernels

// y = x with the dropped elements zeroed, not scaled (ss_dropout.cu)
cudaError_t launch_drop_mask(const uint16_t* x, int64_t n, const DropArgs& drop, uint16_t* y,
                             int num_sms, cudaStream_t stream);

// CTA pairs, 256 x 256 tiles (ss_ffn_pair.cu)
enum GradWhich { kDoX = 1, kDoW = 2 };  // the products of one pair_grads launch
cudaError_t pair_gate_up(const FfnForward& p, int bn, cudaStream_t s);
cudaError_t pair_down(const FfnForward& p, cudaStream_t s);
cudaError_t pair_grad_act(const FfnBackward& p, int bn, cudaStream_t s);  // dG, dU
cudaError_t pair_grads(const FfnBackward& p, int which, cudaStream_t s);

// 128 x (16 to 128) tiles, K split over a cluster (ss_ffn_split.cu)
cudaError_t split_gate_up(const FfnForward& p, const SplitPlan& plan, cudaStream_t s);
cudaError_t split_down(const FfnForward& p, const SplitPlan& plan, cudaStream_t s);
cudaError_t split_grad_act(const FfnBackward& p, const SplitPlan& plan, cudaStream_t s);
cudaError_t split_grad_x(const FfnBackward& p, const SplitPlan& plan, cudaStream_t s);
cudaError_t split_grad_w(const FfnBackward& p, const SplitPlan& plan, cudaStream_t s);

}  // namespace ss
