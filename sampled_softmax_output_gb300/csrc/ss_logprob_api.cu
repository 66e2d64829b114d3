// ss_logprob_api.cu -- the log-probabilities' entry points (include/ss_logprob.h):
// argument checks, the workspace, the launches, and the kernels beside the
// products: the merge of the softmax partials, the coefficients of the backward pass
// and the entries of G at the chosen ids.
#include <algorithm>
#include <cmath>

#include "ss_logprob.cuh"

namespace ss {

namespace {

constexpr size_t kHdrScale = 128;  // byte offset in the header: the scale of dW

size_t up1024(size_t x) { return (x + 1023) / 1024 * 1024; }

struct LogprobLayout {
  size_t part, sorted, z, bin_ends, coef, f, rowfac, hs, dh_part, g, total;
  int64_t ldG;
  int n_parts;
};

// After the header, the forward's softmax partials and sorted ids with their logits,
// or, in the same place, what the backward pass needs: the coefficients, the factors of
// H's and of dH's rows, the scaled H, partial sums of dH, and G. The scale of dW lies
// in the header.
LogprobLayout logprob_layout(int64_t T, int64_t V, int64_t D, bool backward) {
  LogprobLayout L;
  L.ldG = (V + 63) / 64 * 64;
  L.n_parts = static_cast<int>(2 * ((V + kBnLogits - 1) / kBnLogits));
  L.part = L.coef = kHeaderBytes;
  // (a few tokens have partials of another number, kMostFewParts at most)
  const size_t parts = std::max<size_t>(static_cast<size_t>(L.n_parts) * T,
                                        kMostFewParts * std::min<int64_t>(T, kFewTokens));
  L.sorted = L.part + up1024(parts * sizeof(float2));
  L.z = L.sorted + up1024(static_cast<size_t>(T) * SS_MAX_IDS * sizeof(uint32_t));
  L.bin_ends = L.z + up1024(static_cast<size_t>(T) * SS_MAX_IDS * sizeof(float));
  const size_t forward =
      L.bin_ends + up1024(static_cast<size_t>((T + 31) / 32) * L.n_parts * sizeof(uint16_t));
  L.f = L.coef + up1024(static_cast<size_t>(T) * sizeof(float));
  L.rowfac = L.f + up1024(static_cast<size_t>(T) * sizeof(float));
  L.hs = L.rowfac + up1024(static_cast<size_t>(T) * sizeof(float));
  L.dh_part = L.hs + up1024(static_cast<size_t>(T) * D * 2);
  L.g = L.dh_part + up1024(T > 0 ? logprob_part_bytes(T, D) + 32 : 0);
  const size_t both = L.g + up1024(static_cast<size_t>(T) * L.ldG * 2);
  L.total = backward ? std::max(forward, both) : forward;
  return L;
}

ss_status check_logprob_sizes(int64_t T, int64_t V, int64_t D) {
  if (T < 0 || V <= 0 || D <= 0) return SS_ERR_INVALID;
  if (T >= (int64_t(1) << 31) || V > SS_MAX_V || D > SS_MAX_D || D % 64 != 0)
    return SS_ERR_UNSUPPORTED;
  // tiles are counted in 32 bits
  return T * V < (int64_t(1) << 44) ? SS_OK : SS_ERR_UNSUPPORTED;
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool usable(const void* p, uintptr_t a) { return p != nullptr && aligned(p, a); }

ss_status logprob_head(const ss_head* head, LogprobArgs* p) {
  p->cap = 0.f;
  p->tau = 1.f;
  if (head && head->fp8 != 0)
    return head->fp8 == 1 || head->fp8 == 2 ? SS_ERR_UNSUPPORTED : SS_ERR_INVALID;
  if (head && head->cap != 0.f) {
    if (!(head->cap > 0.f) || !std::isfinite(head->cap) || !(head->tau > 0.f) ||
        !std::isfinite(head->tau))
      return SS_ERR_INVALID;
    p->cap = head->cap;
    p->tau = head->tau;
  }
  p->head = head_cap(p->cap, p->tau);
  return SS_OK;
}

// ------------------------------------------------------------- small kernels

// lse[t] from the partials (n, s) of n_parts column groups, and logp = z - lse: of the
// sorted ids' logits z, or (sorted null) in the place of z = logp. A block takes 32
// tokens: warp w folds the partials w, w + 32, ... of its lane's token, the warps' pairs
// meet in shared memory. (16384 tokens, 394 partials: 52 MB in 25 us.)
constexpr int kMergeWarps = 32;

// 2^d for an integer d <= 0; 0 from -127 on
__device__ __forceinline__ float power_of_two(float d) {
  return __int_as_float((static_cast<int>(fmaxf(d, -127.f)) + 127) << 23);
}

// 2^M S += 2^m s
__device__ __forceinline__ void fold(float& M, float& S, float m, float s) {
  if (m == -INFINITY && s == 0.f) return;  // nothing (a row of NaN has a sum of NaN)
  const float nm = fmaxf(M, m);
  S = S * power_of_two(M - nm) + s * power_of_two(m - nm);
  M = nm;
}

// log(2^M S), from S's fraction in [3/4, 3/2) and with log(2) in two parts, so that the
// result is rounded once, in the last addition
__device__ __forceinline__ float log_of(float M, float S) {
  if (!(S > 0.f && S < INFINITY)) return logf(S);  // (no sum is subnormal)
  constexpr float kLn2 = 0.693147180559945309f;
  constexpr float kLn2Lo = static_cast<float>(0.693147180559945309 - double(kLn2));
  const int bits = __float_as_int(S), e = (bits - 0x3f400000) >> 23;
  M += static_cast<float>(e);
  return fmaf(M, kLn2, fmaf(M, kLn2Lo, logf(__int_as_float(bits - e * (1 << 23)))));
}

__global__ void __launch_bounds__(32 * kMergeWarps)
    k_logprob_merge(const float2* __restrict__ part, int n_parts, int T, int K,
                    const int32_t* __restrict__ ids, const uint32_t* __restrict__ sorted,
                    const uint16_t* __restrict__ bin_ends, int bins,
                    const float* __restrict__ z, float* logp, float* __restrict__ lse,
                    int* status) {
  __shared__ float2 red[kMergeWarps][33];
  __shared__ float s_lse[32];
  __shared__ int s_go;
  pdl_enter();
  if (threadIdx.x == 0) s_go = read_status(status) == 0;
  __syncthreads();
  if (!s_go) return;
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 32;
  const int64_t t = t0 + lane;
  float M = -INFINITY, S = 0.f;
  constexpr int kBatch = 8;
  if (t < T)
    for (int c0 = warp; c0 < n_parts; c0 += kMergeWarps * kBatch) {
      float2 q[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + i * kMergeWarps;
        q[i] = c < n_parts ? __ldcs(part + static_cast<int64_t>(c) * T + t)
                           : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) fold(M, S, q[i].x, q[i].y);
    }
  red[warp][lane] = make_float2(M, S);
  __syncthreads();
  // warp w joins token w's pairs: a butterfly, the same order whatever the grid
  {
    float m = red[lane][warp].x, s = red[lane][warp].y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
      const float s2 = __shfl_xor_sync(0xffffffffu, s, o);
      fold(m, s, m2, s2);
    }
    if (lane == 0) {
      const float l = log_of(m, s);
      s_lse[warp] = l;
      if (t0 + warp < T) lse[t0 + warp] = l;
    }
  }
  __syncthreads();
  const int nt = T - t0 < 32 ? static_cast<int>(T - t0) : 32;
  const int64_t at0 = t0 * K;
  if (sorted == nullptr) {
    for (int i = static_cast<int>(threadIdx.x); i < nt * K; i += 32 * kMergeWarps)
      logp[at0 + i] = __ldg(ids + at0 + i) >= 0 ? logp[at0 + i] - s_lse[i / K] : 0.f;
    return;
  }
  const int known = __ldg(bin_ends + (static_cast<int64_t>(blockIdx.x) + 1) * bins - 1);
  for (int i = static_cast<int>(threadIdx.x); i < known; i += 32 * kMergeWarps) {
    const uint32_t e = __ldg(sorted + at0 + i);
    const int row = static_cast<int>((e >> 7) & 31u);
    logp[at0 + row * K + (e >> 12)] = __ldg(z + at0 + i) - s_lse[row];
  }
  if (known < nt * K)
    for (int i = static_cast<int>(threadIdx.x); i < nt * K; i += 32 * kMergeWarps)
      if (__ldg(ids + at0 + i) < 0) logp[at0 + i] = 0.f;
}

// How the backward's two operands are scaled. G's rows are a[t] times probabilities
// and, at the ids, w. Rounded to bf16 as they are, a coefficient that many tokens
// share (those of one preference pair) would put one rounding, up to 2^-8, on all of
// them. So for one id per token, with m the largest |a|,
//   G' = c (P - Y) dz/ds,  dH = (|a| / |c|) (G' W),  dW = m (G'^T (f H)),  |a| = m f |c|
// where f is a power of two, which leaves H exact, and 1 <= |c| < 2; tokens of
// coefficient m have c = 1. Where that would round the entry at the id, c (1 - P)
// dz/ds, by more than kMostRounding, c is the number nearest 1 that makes it a bf16
// number and f takes the rest: H's own rounding is as large but differs from element to
// element. (32 tokens of one pair: dH and dW, as bf16, 3.0e-3 off without, 1.7e-3 and
// 2.1e-3 with. 16384 tokens of a policy loss: 2.4e-3 without, 1.8e-3 and 2.1e-3 with.)
// With several ids per token G's entries round independently: f = 1, G' = G.
constexpr float kMostRounding = 0x1.6p-10f;

// dz/ds of a chosen id, whose z is logp + lse: off by some 1e-6, beside a slope of up to
// cap / (4 tau) by 4e-6 / cap of it, which must be little beside G's rounding.
constexpr float kLeastCap = 0x1p-6f;

__device__ __forceinline__ float head_slope(float z, const HeadCap& h) {
  return h.cap > 0.f ? z * ((h.cap - z) * h.icap_tau) : 1.f;
}

// K = 1: the largest |w| among tokens first, first + step, ... and whether an id is bad.
__device__ __forceinline__ float top_coef(const float* __restrict__ dlogp,
                                          const int32_t* __restrict__ ids, int64_t first,
                                          int64_t step, int T, int V, bool& bad) {
  float top = 0.f;
#pragma unroll 4
  for (int64_t t = first; t < T; t += step) {
    const int id = __ldg(ids + t);
    const float w = __ldg(dlogp + t);
    bad |= id < -1 || id >= V;
    if (id >= 0) top = fmaxf(top, fabsf(w));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

struct CoefArgs {
  const float* dlogp;
  const int32_t* ids;
  const float *logp, *lse;
  HeadCap head;
  float* coef;
  uint32_t* entry;
  float* rowfac;
  const uint16_t* H;
  uint16_t* Hs;
  int D;
};

// Hs[t] = f H[t], a warp's work: 0 for f = 0 (not 0 times an infinity or a NaN of H)
__device__ __forceinline__ void scale_row(const uint16_t* __restrict__ H,
                                          uint16_t* __restrict__ Hs, int64_t t, int D, float f,
                                          int lane) {
  const uint4* src = reinterpret_cast<const uint4*>(H + t * D);
  uint4* dst = reinterpret_cast<uint4*>(Hs + t * D);
  for (int c = lane; c < D / 8; c += 32) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (f != 0.f) {
      v = __ldg(src + c);
      if (f != 1.f) {
        uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = pack_bf16x2(__uint_as_float(x[i] << 16) * f,
                             __uint_as_float(x[i] & 0xffff0000u) * f);
        v = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
    dst[c] = v;
  }
}

// K = 1, a warp for token t: coef[t] = c, with the sign of a; rowfac[t] = |a| / |c|, 0
// where a is; entry[t], G's at the id as bf16; Hs[t] = f H[t].
__device__ __forceinline__ void scale_coef(const CoefArgs& p, int64_t t, float top, int lane) {
  const float w = __ldg(p.ids + t) >= 0 ? __ldg(p.dlogp + t) : 0.f;
  const float l = __ldg(p.logp + t), z = l + __ldg(p.lse + t);
  float c = 0.f, ft = 0.f, rf = 0.f, g = 0.f;
  if (w != 0.f) {  // (a NaN too)
    const float size = fabsf(w), x = size / top;
    // the power of two below x; x itself where it is none or no normal number
    ft = __uint_as_float(__float_as_uint(x) & 0x7f800000u);
    if (!(ft > 0.f && ft <= 1.f)) ft = x;
    c = x > 0.f ? x / ft : 1.f;  // (beside an infinite coefficient x is 0)
    const float q = -expm1f(l) * head_slope(z, p.head);
    g = c * q;
    const auto rounded = [](float v) {
      return __uint_as_float(static_cast<uint32_t>(bf16_bits(v)) << 16);
    };
    if (x > 0.f && !(fabsf(rounded(g) - g) <= kMostRounding * fabsf(g))) {
      c = rounded(q) / q;
      if (!(c > 0.5f && c < 2.f)) c = 1.f;  // (q is no normal number)
      ft = x / c;
      g = c * q;
    }
    rf = size / c;
    if (w > 0.f) c = -c;
    else g = -g;
  }
  if (lane == 0) {
    p.coef[t] = c;
    p.rowfac[t] = rf;
    p.entry[t] = bf16_bits(g);
  }
  scale_row(p.H, p.Hs, t, p.D, ft, lane);
}

// Up to kOneKernelTokens every block finds m by itself, from 8 bytes a token, and scales
// its tokens; beyond, a kernel for each. (With the entries written over G and H scaled in
// a kernel of their own behind G's, the backward pass of 256, 1024 and 4096 tokens took
// 73, 167 and 556 us for 71, 164 and 552.)
constexpr int kCoefThreads = 256, kOneKernelTokens = 4096;

__global__ void __launch_bounds__(kCoefThreads)
    k_logprob_coef_one(const CoefArgs p, int T, int V, float* __restrict__ scale, int* status) {
  __shared__ float s_top[kCoefThreads / 32];
  __shared__ int s_go;
  pdl_enter();
  if (threadIdx.x == 0) s_go = read_status(status) == 0;
  __syncthreads();
  if (!s_go) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  bool bad = false;
  float top = top_coef(p.dlogp, p.ids, threadIdx.x, kCoefThreads, T, V, bad);
  if (bad) set_status(status, SS_ERR_TARGET_RANGE);
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  for (int w = 0; w < kCoefThreads / 32; ++w) top = fmaxf(top, s_top[w]);
  if (blockIdx.x == 0 && threadIdx.x == 0) *scale = top;
  const int step = static_cast<int>(gridDim.x) * (kCoefThreads / 32);
  for (int t = static_cast<int>(blockIdx.x) * (kCoefThreads / 32) + warp; t < T; t += step)
    scale_coef(p, t, top, lane);
}

// *scale, 0 before, as the bits of a number that is not negative
__global__ void __launch_bounds__(256) k_logprob_top(const CoefArgs p, int T, int V,
                                                     uint32_t* scale, int* status) {
  pdl_enter();
  if (read_status(status) != 0) return;
  bool bad = false;
  const float top = top_coef(p.dlogp, p.ids, blockIdx.x * int64_t(256) + threadIdx.x,
                             int64_t(gridDim.x) * 256, T, V, bad);
  if (bad) set_status(status, SS_ERR_TARGET_RANGE);
  if ((threadIdx.x & 31) == 0 && top > 0.f) atomicMax(scale, __float_as_uint(top));
}

__global__ void __launch_bounds__(256) k_logprob_scale(const CoefArgs p, int T,
                                                       const float* scale, int* status) {
  pdl_enter();
  if (read_status(status) != 0) return;
  const float top = *scale;
  for (int64_t t = blockIdx.x * int64_t(8) + threadIdx.x / 32; t < T; t += int64_t(gridDim.x) * 8)
    scale_coef(p, t, top, threadIdx.x & 31);
}

// K > 1: coef[t] = -sum_k w[t, k], and f[t] = 1 or 0: whether any w is not 0. A warp
// per token.
__global__ void __launch_bounds__(256) k_logprob_coef(const float* __restrict__ dlogp,
                                                      const int32_t* __restrict__ ids, int K,
                                                      int T, int V, float* __restrict__ coef,
                                                      float* __restrict__ f, int* status) {
  pdl_enter();
  if (read_status(status) != 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
  for (int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + threadIdx.x / 32; t < T;
       t += step) {
    float sum = 0.f;
    bool some = false, bad = false;
    for (int k = lane; k < K; k += 32) {
      const int id = __ldg(ids + t * K + k);
      bad |= id < -1 || id >= V;
      const float w = id >= 0 ? __ldg(dlogp + t * K + k) : 0.f;
      some |= w != 0.f;
      sum -= w;
    }
    if (bad) set_status(status, SS_ERR_TARGET_RANGE);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    some = __any_sync(0xffffffffu, some);
    if (lane == 0) {
      coef[t] = sum;
      f[t] = some ? 1.f : 0.f;
    }
  }
}

// K > 1: G[t, ids[t, k]], in the place of what the product wrote there, and f H. The sum
// of an entry is rounded once; of several equal ids the first writes it. A warp per
// token.
__global__ void __launch_bounds__(256) k_logprob_patch(
    const float* __restrict__ dlogp, const int32_t* __restrict__ ids,
    const float* __restrict__ logp, const float* __restrict__ lse,
    const float* __restrict__ coef, const float* __restrict__ f, int K, int T, int V, int D,
    HeadCap head, const uint16_t* __restrict__ H, uint16_t* __restrict__ Hs,
    uint16_t* __restrict__ G, int64_t ldG, int* status) {
  __shared__ __align__(16) int s_id[8][SS_MAX_IDS];
  __shared__ float s_w[8][SS_MAX_IDS];
  static_assert(SS_MAX_IDS % 4 == 0, "four ids at a time");
  pdl_enter();
  if (read_status(status) != 0) return;  // no barrier of the block follows
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
  for (int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + warp; t < T; t += step) {
    const float a = __ldg(coef + t);
    const int K4 = (K + 3) / 4 * 4;
    for (int k = lane; k < K4; k += 32) {
      const int id = k < K ? __ldg(ids + t * K + k) : -1;
      s_id[warp][k] = id < V ? id : -1;
      s_w[warp][k] = id >= 0 ? __ldg(dlogp + t * K + k) : 0.f;
    }
    __syncwarp();
    for (int k = lane; k < K; k += 32) {
      const int id = s_id[warp][k];
      if (id < 0) continue;
      float w = s_w[warp][k];
      int equal = 0;
      for (int j = 0; j < K4; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(&s_id[warp][j]);
        equal += (v.x == id) + (v.y == id) + (v.z == id) + (v.w == id);
      }
      if (equal > 1) {  // rare: the sum of them all, written by the first
        bool first = true;
        w = 0.f;
        for (int j = 0; j < K; ++j)
          if (s_id[warp][j] == id) {
            first = first && j >= k;
            w += s_w[warp][j];
          }
        if (!first) continue;
      }
      const float l = __ldg(logp + t * K + k);
      const float g = a != 0.f ? fmaf(a, expf(l), w) : w;
      G[t * ldG + id] =
          g != 0.f ? bf16_bits(g * head_slope(l + __ldg(lse + t), head)) : uint16_t(0);
    }
    __syncwarp();
    scale_row(H, Hs, t, D, __ldg(f + t), lane);
  }
}

int warps_grid(int64_t items, int num_sms) {
  const int64_t blocks = (items + 7) / 8, most = static_cast<int64_t>(num_sms) * 8;
  return static_cast<int>(std::min(blocks, most));
}

}  // namespace

}  // namespace ss

using namespace ss;

extern "C" {

size_t ss_logprob_workspace_size(int64_t T, int64_t V, int64_t D, int backward) {
  return check_logprob_sizes(T, V, D) == SS_OK ? logprob_layout(T, V, D, backward != 0).total : 0;
}

ss_status ss_logprob_forward(const uint16_t* H, const uint16_t* W, const int32_t* ids, int64_t K,
                             int64_t T, int64_t V, int64_t D, const ss_head* head, float* logp,
                             float* lse, void* workspace, size_t workspace_bytes,
                             ss_stream stream) {
  LogprobArgs p = {};
  ss_status st = check_logprob_sizes(T, V, D);
  if (st == SS_OK) st = logprob_head(head, &p);
  if (st != SS_OK) return st;
  if (K < 1) return SS_ERR_INVALID;
  if (K > SS_MAX_IDS) return SS_ERR_UNSUPPORTED;
  if (!usable(workspace, 16) || !usable(W, 16) ||
      (T > 0 && (!usable(H, 16) || !usable(ids, 4) || !usable(logp, 4) || !usable(lse, 4))))
    return SS_ERR_INVALID;
  const LogprobLayout L = logprob_layout(T, V, D, false);
  if (workspace_bytes < L.total) return SS_ERR_WORKSPACE;
  if (T == 0) return SS_OK;
  p.num_sms = current_num_sms();
  if (p.num_sms <= 0)
    return record_failure("cudaGetDevice/cudaDeviceGetAttribute", cudaGetLastError());
  char* ws = static_cast<char*>(workspace);
  p.H = H, p.W = W;
  p.T = static_cast<int>(T), p.V = static_cast<int>(V), p.D = static_cast<int>(D);
  p.status = reinterpret_cast<int*>(ws);
  float2* part = reinterpret_cast<float2*>(ws + L.part);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int iK = static_cast<int>(K);
  cudaError_t e;
  uint32_t* sorted = reinterpret_cast<uint32_t*>(ws + L.sorted);
  uint16_t* bin_ends = reinterpret_cast<uint16_t*>(ws + L.bin_ends);
  float* z = reinterpret_cast<float*>(ws + L.z);
  const int few = logprob_few_parts(T, V, p.num_sms);
  if (few) {
    StageTrace trace(s, "gemm_forward_lse");
    e = launch_logprob_few(p, iK, ids, few, part, logp, s);
  } else {
    {
      StageTrace trace(s, "bin_ids");
      e = launch_bin_ids(p, ids, iK, L.n_parts, sorted, bin_ends, s);
    }
    if (e != cudaSuccess) return record_failure("launch k_bin_ids", e);
    StageTrace trace(s, "gemm_forward_lse");
    e = launch_logprob_partials(p, iK, sorted, bin_ends, part, z, s);
  }
  if (e != cudaSuccess) return record_failure("launch gemm_forward_lse", e);
  {
    StageTrace trace(s, "logprob_merge");
    e = launch_pdl(k_logprob_merge, dim3(static_cast<unsigned>((T + 31) / 32)),
                   dim3(32 * kMergeWarps), 0, s, part, few ? few : L.n_parts, p.T, iK, ids,
                   few ? nullptr : sorted, bin_ends, L.n_parts, z, logp, lse, p.status);
  }
  return e == cudaSuccess ? SS_OK : record_failure("launch k_logprob_merge", e);
}

ss_status ss_logprob_backward(const float* dlogp, const uint16_t* H, const uint16_t* W,
                              const int32_t* ids, const float* logp, const float* lse, int64_t K,
                              int64_t T, int64_t V, int64_t D, const ss_head* head, int dw_dtype,
                              int accumulate, uint16_t* dH, void* dW, void* workspace,
                              size_t workspace_bytes, ss_stream stream) {
  LogprobArgs p = {};
  ss_status st = check_logprob_sizes(T, V, D);
  if (st == SS_OK) st = logprob_head(head, &p);
  if (st != SS_OK) return st;
  if (K < 1 || (dw_dtype != SS_BF16 && dw_dtype != SS_FP32) ||
      (accumulate != 0 && accumulate != 1))
    return SS_ERR_INVALID;
  if (K > SS_MAX_IDS || (p.cap > 0.f && p.cap < kLeastCap)) return SS_ERR_UNSUPPORTED;
  if (!usable(workspace, 16) || !usable(W, 16) || !usable(dW, 16) ||
      (T > 0 && (!usable(H, 16) || !usable(dH, 16) || !usable(ids, 4) || !usable(dlogp, 4) ||
                 !usable(logp, 4) || !usable(lse, 4))))
    return SS_ERR_INVALID;
  const LogprobLayout L = logprob_layout(T, V, D, true);
  if (workspace_bytes < L.total) return SS_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (accumulate) return SS_OK;
    const cudaError_t e = cudaMemsetAsync(
        dW, 0, static_cast<size_t>(V) * D * (dw_dtype == SS_FP32 ? 4 : 2), s);
    return e == cudaSuccess ? SS_OK : record_failure("cudaMemsetAsync(dW)", e);
  }
  p.num_sms = current_num_sms();
  if (p.num_sms <= 0)
    return record_failure("cudaGetDevice/cudaDeviceGetAttribute", cudaGetLastError());
  char* ws = static_cast<char*>(workspace);
  p.H = H, p.W = W;
  p.T = static_cast<int>(T), p.V = static_cast<int>(V), p.D = static_cast<int>(D);
  p.status = reinterpret_cast<int*>(ws);
  float* coef = reinterpret_cast<float*>(ws + L.coef);
  float* rowfac = reinterpret_cast<float*>(ws + L.rowfac);
  float* f = reinterpret_cast<float*>(ws + L.f);            // K > 1
  uint32_t* entry = reinterpret_cast<uint32_t*>(ws + L.f);  // K = 1
  float* scale = reinterpret_cast<float*>(ws + kHdrScale);
  uint16_t* Hs = reinterpret_cast<uint16_t*>(ws + L.hs);
  uint16_t* G = reinterpret_cast<uint16_t*>(ws + L.g);
  // (the workspace itself may lie between two 32-byte boundaries)
  float* part = reinterpret_cast<float*>(
      (reinterpret_cast<uintptr_t>(ws + L.dh_part) + 31) / 32 * 32);
  const int iK = static_cast<int>(K), grid = warps_grid(T, p.num_sms);
  cudaError_t e;
  {
    StageTrace trace(s, "logprob_coef");
    const CoefArgs c{dlogp, ids, logp, lse, p.head, coef, entry, rowfac, H, Hs, p.D};
    if (iK > 1) {
      e = launch_pdl(k_logprob_coef, dim3(grid), dim3(256), 0, s, dlogp, ids, iK, p.T, p.V, coef,
                     f, p.status);
    } else if (T <= kOneKernelTokens) {
      e = launch_pdl(k_logprob_coef_one, dim3(grid), dim3(kCoefThreads), 0, s, c, p.T, p.V, scale,
                     p.status);
    } else {
      const dim3 blocks(static_cast<unsigned>(std::min((T + 255) / 256, int64_t(p.num_sms) * 4)));
      e = cudaMemsetAsync(scale, 0, sizeof *scale, s);
      if (e == cudaSuccess)
        e = launch_pdl(k_logprob_top, blocks, dim3(256), 0, s, c, p.T, p.V,
                       reinterpret_cast<uint32_t*>(scale), p.status);
      if (e == cudaSuccess)
        e = launch_pdl(k_logprob_scale, dim3(grid), dim3(256), 0, s, c, p.T,
                       static_cast<const float*>(scale), p.status);
    }
  }
  if (e != cudaSuccess) return record_failure("launch k_logprob_coef", e);
  {
    StageTrace trace(s, "gemm_softmax_grad");
    e = launch_logprob_g(p, coef, lse, iK == 1 ? ids : nullptr, entry, G, L.ldG, s);
  }
  if (e != cudaSuccess) return record_failure("launch gemm_softmax_grad", e);
  if (iK > 1) {
    StageTrace trace(s, "logprob_patch");
    e = launch_pdl(k_logprob_patch, dim3(grid), dim3(256), 0, s, dlogp, ids, logp, lse, coef, f,
                   iK, p.T, p.V, p.D, p.head, H, Hs, G, L.ldG, p.status);
  }
  if (e != cudaSuccess) return record_failure("launch k_logprob_patch", e);
  {
    StageTrace trace(s, "gemm_grads");
    e = launch_logprob_grads(p, G, L.ldG, Hs, iK == 1 ? rowfac : nullptr,
                             iK == 1 ? scale : nullptr, part, dH, dW, dw_dtype == SS_FP32,
                             accumulate, s);
  }
  return e == cudaSuccess ? SS_OK : record_failure("launch gemm_grads", e);
}

}  // extern "C"
