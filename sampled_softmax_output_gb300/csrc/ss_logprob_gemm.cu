// ss_logprob_gemm.cu -- the logits again, for the backward pass of the head's
// log-probabilities: G = (a exp(z - lse)) dz/ds with z = H W^T (M = T, N = V, K = D),
// on the GEMM cores of ss_gemm.cuh and ss_gemm2.cuh.
#include "ss_gemm.cuh"
#include "ss_gemm2.cuh"
#include "ss_logprob.cuh"

namespace ss {

namespace {

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(v)) : "memory");
}

// The logits of a tile become the rows a[t] exp(z - lse) dz/ds of G, a
// coefficient of either sign for each row: exp(z - (lse - log|a|)) with the
// sign put in afterwards. A row of coefficient 0 is 0 whatever its logits are. With one
// id per token its entry, which is more than that, goes over it on the way out.
// Two column groups of four warps, each with a 16 KB staging buffer that holds
// a 64-column quarter in the swizzled layout of G's tensor map.
template <bool CAP>
struct EpiCoef {
  static constexpr int kStageBytes = 2 * 16384;
  static constexpr bool kKeepOperands = true;
  static constexpr bool kSelfRelease = true;
  struct Params {
    CUtensorMap tmG;  // G [T, V] bf16, box 64 x 128, 128-byte swizzle
    int T, V;
    const float* coef;
    const float* lse;
    const int32_t* ids;     // null: no entries of their own
    const uint32_t* entry;  // bf16 at column ids[t]
    HeadCap head;
  };
  __device__ static void begin(const Params&, EpiState&) {}
  __device__ static void finish(const Params&, EpiState& es) {
    if ((es.ep_tid & 127) == 0) bulk_wait<0>();
  }
  template <int BN, int NCG, class Rel>
  __device__ static void apply(const Params& p, int mt, int nt, int row, uint32_t taddr,
                               EpiState& es, int cg, Rel&& release) {
    static_assert(NCG == 2 && BN == 256, "two column groups of two 64-column quarters");
    constexpr int CPG = BN / 32 / NCG;
    const int bar = 1 + 2 * cg;
    const bool leader = (es.ep_tid & 127) == 0;
    const int t = mt * BM + row;
    const bool valid = t < p.T;
    const float a = valid ? __ldg(p.coef + t) : 0.f;
    const uint32_t keep = a != 0.f ? 0xffffffffu : 0u;
    const uint32_t sgn = a < 0.f ? 0x80008000u : 0u;
    const float off2 = keep ? fmaf(__ldg(p.lse + t), kLog2e, -log2f(fabsf(a))) : 0.f;
    const int j0 = nt * BN;
    const int own = valid && p.ids ? __ldg(p.ids + t) - j0 : -1;  // its column of the tile
    const uint32_t entry = own >= 0 && own < BN ? __ldg(p.entry + t) : 0u;
    const int ncols = min(BN, p.V - j0);
    const uint32_t r7 = static_cast<uint32_t>(row & 7);
    const uint32_t buf = es.stage + static_cast<uint32_t>(cg) * 16384u;
    const uint32_t rowbase = buf + static_cast<uint32_t>(row) * 128u;
    for_tmem_chunks<CPG>(taddr, cg * CPG, [&](const uint32_t(&v)[32], int i) {
      const int jc = (cg * CPG + i) * 32;  // column of the tile
      if (jc >= ncols) return;             // uniform: depends on the tile only
      const int h = i & 1;                 // half of the quarter
      if (h == 0) {
        // the store that last used this buffer must have read it
        if (es.rounds >= 1 && leader) bulk_wait_read<0>();
        named_bar_sync(bar, 128);
      }
      uint32_t pk[16];
      const uint64_t noff = f32x2(-off2, -off2);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint64_t x = f32x2_bits(v[2 * k], v[2 * k + 1]);
        float y0, y1, g0, g1;
        if constexpr (CAP) {
          // with w = 1 / (1 + exp(-s / tau)): z = cap w, dz/ds = (cap / tau) w (1 - w); two
          // logits to an operation (814 us instead of 895 at T 16384, D 768)
          const auto both = [](float c) { return f32x2(c, c); };
          f32x2_split(mul_f32x2(x, both(-p.head.k1)), y0, y1);
          f32x2_split(add_f32x2(f32x2(ex2_approx(y0), ex2_approx(y1)), both(1.f)), y0, y1);
          const uint64_t w = f32x2(rcp_approx(y0), rcp_approx(y1));
          f32x2_split(fma_f32x2(w, both(p.head.cap * kLog2e), noff), y0, y1);
          const uint64_t slope = mul_f32x2(mul_f32x2(w, fma_f32x2(w, both(-1.f), both(1.f))),
                                           both(p.head.cap * (p.head.cap * p.head.icap_tau)));
          f32x2_split(mul_f32x2(f32x2(ex2_approx(y0), ex2_approx(y1)), slope), g0, g1);
        } else {
          f32x2_split(fma_f32x2(x, f32x2(kLog2e, kLog2e), noff), y0, y1);
          g0 = ex2_approx(y0);
          g1 = ex2_approx(y1);
        }
        pk[k] = (pack_bf16x2(g0, g1) ^ sgn) & keep;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t ci = static_cast<uint32_t>(h * 4 + w);
        st_shared_v4(rowbase + ((ci ^ r7) << 4), pk[4 * w], pk[4 * w + 1], pk[4 * w + 2],
                     pk[4 * w + 3]);
      }
      if (own >= jc && own < jc + 32) {
        const uint32_t c = static_cast<uint32_t>(h * 32 + own - jc);
        st_shared_u16(rowbase + (((c >> 3) ^ r7) << 4) + (c & 7u) * 2u, entry);
      }
      if (h == 1 || jc + 32 >= ncols) {  // the quarter is complete: store it
        fence_proxy_async_smem();
        named_bar_sync(bar, 128);
        if (leader) {
          tma_store_2d_hint(&p.tmG, buf, j0 + jc - 32 * h, mt * BM, l2_evict_first());
          bulk_commit();
        }
        ++es.rounds;
      }
    }, release);
  }
};

// Units walk groups of this many rows column tile by column tile, so that W is read from
// memory once per group while G streams out (row by row, W came 7 times: V 50304, T 16384,
// D 768 815 us for 767; T 8192, D 2048 1120 for 930).
constexpr int kGroupRows = 8192;

template <bool CAP>
cudaError_t coef_gemm(const LogprobArgs& p, const float* coef, const float* lse,
                      const int32_t* ids, const uint32_t* entry, uint16_t* G, int64_t ldG,
                      cudaStream_t s) {
  CUtensorMap tH, tW;
  typename EpiCoef<CAP>::Params ep;
  const uint64_t row = static_cast<uint64_t>(p.D) * 2;
  const int n_tiles = (p.V + kBnLogits - 1) / kBnLogits;
  const bool pairs = softmax_grad_on_pairs(p.T, p.V, p.num_sms);
  if (!make_bf16_map(&tH, p.H, p.D, p.T, row, 64, 128) ||
      !make_bf16_map(&tW, p.W, p.D, p.V, row, 64, pairs ? kBnLogits / 2 : kBnLogits) ||
      !make_bf16_map(&ep.tmG, G, p.V, p.T, static_cast<uint64_t>(ldG) * 2, 64, 128))
    return cudaErrorInvalidValue;
  ep.T = p.T;
  ep.V = p.V;
  ep.coef = coef;
  ep.lse = lse;
  ep.ids = ids;
  ep.entry = entry;
  ep.head = p.head;
  if (pairs) {
    GemmShape shp{(p.T + 2 * BM - 1) / (2 * BM), n_tiles, p.D / BK, 0, 0, nullptr,
                  kGroupRows / (2 * BM)};
    return launch_gemm2<kBnLogits, 6, false, false, EpiCoef<CAP>, 8>(tH, tW, shp, ep, p.status,
                                                                     p.num_sms, s);
  }
  GemmShape shp{(p.T + BM - 1) / BM, n_tiles, p.D / BK, 0, 0, nullptr, kGroupRows / BM};
  return launch_gemm<kBnLogits, 4, false, false, EpiCoef<CAP>, 8>(tH, tW, shp, ep, p.status,
                                                                  p.num_sms, s);
}

}  // namespace

cudaError_t launch_logprob_g(const LogprobArgs& p, const float* coef, const float* lse,
                             const int32_t* ids, const uint32_t* entry, uint16_t* G, int64_t ldG,
                             cudaStream_t s) {
  return p.cap > 0.f ? coef_gemm<true>(p, coef, lse, ids, entry, G, ldG, s)
                     : coef_gemm<false>(p, coef, lse, ids, entry, G, ldG, s);
}

}  // namespace ss
