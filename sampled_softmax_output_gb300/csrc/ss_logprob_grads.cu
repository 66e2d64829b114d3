// ss_logprob_grads.cu -- the two gradients of the head's log-probabilities in one
// launch of CTA pairs (the protocol of ss_gemm2.cuh):
//   dH = G W     (M = T, N = D, K = V), rows times their factor
//   dW = G^T Hs  (M = V, N = D, K = T), every vocabulary row, times one scale
// With few tokens dH has a handful of 256 x 256 tiles and the whole vocabulary to sum
// over: then K is cut into slices, whose sums k_join_dh adds in their order (the same
// bits every time). The tiles of dW keep the other pairs busy meanwhile; a tile of
// either length goes to the pair that is free first (deal_units of ss_ffn_plan.h).
#include <algorithm>
#include <type_traits>

#include "ss_ffn.cuh"
#include "ss_gemm.cuh"
#include "ss_gemm2.cuh"
#include "ss_logprob.cuh"

namespace ss {

namespace {

constexpr int kBN = 256;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
// a 16 KB buffer for each column group's stores of dW beside the ring
constexpr int kStageBytes = 2 * 16384;
using L = Gemm2Smem<kBN, kStages, kStageBytes>;

struct GradArgs {
  CUtensorMap tmDw;        // dW [V, D] as rows of two-byte words, fp32 too
  CUtensorMap tmGk, tmW;   // dH: G [T, V] by rows, W [V, D]
  CUtensorMap tmGm, tmHs;  // dW: G [T, V] by columns, Hs [T, D]
  UnitDeal deal;           // units 0 .. n_dw - 1: dW's tiles, then dH's tiles by slice
  int n_dw, n_nt, m_dh, slices, kb_dw, kb_dh;
  int T, V, D;
  uint16_t* dH;
  float* part;          // slices > 1: [slices][T][D] sums of dH
  const float* rowfac;  // null: 1
  void* dW;
  const float* scale;   // null: 1
  int accumulate;
  int* status;
};

struct GradUnit {
  int dw, mt, nt, slice, kb0, kb1;
};

__device__ __forceinline__ GradUnit grad_unit(const GradArgs& p, int u) {
  GradUnit g;
  g.dw = u < p.n_dw;
  const int v = g.dw ? u : u - p.n_dw;
  g.nt = v % p.n_nt;
  const int r = v / p.n_nt;
  g.slice = g.dw ? 0 : r / p.m_dh;
  g.mt = g.dw ? r : r % p.m_dh;
  g.kb0 = g.dw ? 0 : static_cast<int>(static_cast<int64_t>(p.kb_dh) * g.slice / p.slices);
  g.kb1 = g.dw ? p.kb_dw
               : static_cast<int>(static_cast<int64_t>(p.kb_dh) * (g.slice + 1) / p.slices);
  return g;
}

// 32 columns of a row of dW, added to what is there
template <bool FP32>
__device__ __forceinline__ void add_dw(const GradArgs& p, size_t at, const uint32_t (&r)[32],
                                       float f) {
  if constexpr (FP32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.dW) + at);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float4 old = dst[k];
      dst[k] = make_float4(fmaf(__uint_as_float(r[4 * k]), f, old.x),
                           fmaf(__uint_as_float(r[4 * k + 1]), f, old.y),
                           fmaf(__uint_as_float(r[4 * k + 2]), f, old.z),
                           fmaf(__uint_as_float(r[4 * k + 3]), f, old.w));
    }
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dW) + at);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 x = dst[k];
      const uint32_t old[4] = {x.x, x.y, x.z, x.w};
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16x2(fmaf(__uint_as_float(r[8 * k + 2 * e]), f, bf16_lo(old[e])),
                           fmaf(__uint_as_float(r[8 * k + 2 * e + 1]), f, bf16_hi(old[e])));
      dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <bool FP32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_logprob_grads(const __grid_constant__ GradArgs p) {
  pdl_enter();
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_go;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  GemmCtrl* ctrl = reinterpret_cast<GemmCtrl*>(smem + L::CTRL_OFFSET);
  const uint32_t tiles = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const PairShare share = share_of(p.deal, static_cast<int>(blockIdx.x >> 1),
                                   static_cast<int>(gridDim.x >> 1));
  const int units = share.count();

  // both CTAs of a pair take the same decision
  if (threadIdx.x == 0) s_go = read_status(p.status) == 0;
  cluster_sync_all();
  if (threadIdx.x == 0)
    s_go = s_go && ld_shared_cluster_u32(mapa_shared(smem_u32(&s_go), rank ^ 1u));
  cluster_sync_all();
  if (!s_go) return;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->tempty[b], 2 * kEpiWarps);
    }
    mbar_init(&ctrl->drain, 1);
    ctrl->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&p.tmGk);
    tma_prefetch_map(&p.tmW);
    tma_prefetch_map(&p.tmGm);
    tma_prefetch_map(&p.tmHs);
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctrl->tmem_base, 2 * kBN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = ctrl->tmem_base;
  volatile int* abort_flag = &ctrl->abort_flag;

  if (warp == 0) {
    // ------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_ph = 0;
      bool ok = true;
      const uint64_t keep = l2_evict_last();  // W and Hs are re-read by every row tile
      // (a loop for each kind of unit, here and below: what this one thread decides per
      // k-block, both CTAs' tensor cores wait for; T 3001, D 1024, V 24576: 177 us, with
      // the kind asked for at every copy and MMA 202)
      auto load = [&](const GradUnit& g, const CUtensorMap* ma, const CUtensorMap* mb, auto dw) {
        const int m0 = g.mt * 2 * BM + static_cast<int>(rank) * BM;
        const int n0 = g.nt * kBN + static_cast<int>(rank) * (kBN / 2);
        for (int kb = g.kb0; kb < g.kb1; ++kb) {
          if (!mbar_wait(&ctrl->empty[s], ph ^ 1u, abort_flag, p.status)) return false;
          const uint32_t fb_local = smem_u32(&ctrl->full[s]);
          if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * L::STAGE_BYTES);
          const uint32_t fb = rank == 0 ? fb_local : mapa_shared(fb_local, 0);
          const uint32_t a_dst = tiles + s * L::STAGE_BYTES;
          const uint32_t b_dst = a_dst + L::A_BYTES;
          if constexpr (decltype(dw)::value) {
            tma_load_2d_pair(a_dst, ma, fb, m0, kb * BK);
            tma_load_2d_pair(a_dst + 8192, ma, fb, m0 + 64, kb * BK);
          } else {
            tma_load_2d_pair(a_dst, ma, fb, kb * BK, m0);
          }
          tma_load_2d_pair_hint(b_dst, mb, fb, n0, kb * BK, keep);
          tma_load_2d_pair_hint(b_dst + 8192, mb, fb, n0 + 64, kb * BK, keep);
          issued |= 1u << s;
          issued_ph = (issued_ph & ~(1u << s)) | (ph << s);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        return true;
      };
      for (int i = 0; ok && i < units; ++i) {
        const GradUnit g = grad_unit(p, share.unit(i));
        ok = g.dw ? load(g, &p.tmGm, &p.tmHs, std::true_type{})
                  : load(g, &p.tmGk, &p.tmW, std::false_type{});
      }
      if (rank == 0) {
        for (int i = 0; i < kStages; ++i)
          if ((issued >> i) & 1u) mbar_drain(&ctrl->full[i], (issued_ph >> i) & 1u, p.status);
      } else if (!ok) {
        // aborted: the peer cannot observe the leader's barriers; its copies in
        // flight get a bounded moment to land before shared memory goes
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (leader)
    if (lane == 0 && rank == 0) {
      int s = 0, b = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      auto multiply = [&](const GradUnit& g, uint32_t d_tmem, auto dw) {
        constexpr bool kDw = decltype(dw)::value;
        constexpr uint32_t idesc = idesc_bf16_f32(2 * BM, kBN, kDw, true);
        for (int kb = g.kb0; kb < g.kb1; ++kb) {
          if (!mbar_wait(&ctrl->full[s], ph, abort_flag, p.status)) return false;
          tc_fence_after();
          const uint32_t a_addr = tiles + s * L::STAGE_BYTES;
          const uint32_t b_addr = a_addr + L::A_BYTES;
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k)
            mma_bf16_pair(d_tmem,
                          kDw ? sdesc_sw128(a_addr + k * 2048, 8192, 1024)
                              : sdesc_sw128(a_addr + k * 32, 16, 1024),
                          sdesc_sw128(b_addr + k * 2048, 8192, 1024), idesc,
                          (kb > g.kb0 || k > 0) ? 1u : 0u);
          mma_commit_pair(&ctrl->empty[s], 0x3);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        return true;
      };
      for (int i = 0; ok && i < units; ++i) {
        const GradUnit g = grad_unit(p, share.unit(i));
        if (!mbar_wait(&ctrl->tempty[b], aph ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * kBN);
        ok = g.dw ? multiply(g, d_tmem, std::true_type{}) : multiply(g, d_tmem, std::false_type{});
        if (!ok) break;
        mma_commit_pair(&ctrl->tfull[b], 0x3);
        if (++b == 2) {
          b = 0;
          aph ^= 1u;
        }
      }
      mma_commit_pair(&ctrl->drain, 0x1);
      mbar_drain(&ctrl->drain, 0, p.status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;         // TMEM lane quarter this warp may access
    const int cg = (warp - 2) / 4;  // its half of the tile's columns
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + cg * (kBN / 2);
    const float scale = p.scale ? __ldg(p.scale) : 1.f;
    const int bar = 1 + 2 * cg;  // the column group's barrier
    const bool leader = threadIdx.x - 64 - cg * 128 == 0;
    const uint32_t buf = tiles + L::EPI_OFFSET + static_cast<uint32_t>(cg) * 16384u;
    const uint32_t rowbase = buf + static_cast<uint32_t>(q * 32 + lane) * 128u;
    const uint32_t r7 = static_cast<uint32_t>(lane & 7);
    int b = 0;
    uint32_t aph = 0;
    for (int i = 0; i < units; ++i) {
      const bool ok = mbar_wait(&ctrl->tfull[b], aph, abort_flag, p.status);
      // the warps stop together: they meet at the groups' barriers
      const bool mine = __all_sync(0xffffffffu, ok);
      if (lane == 0) ctrl->vote[i & 1][warp - 2] = mine ? 1 : 0;
      named_bar_sync(2, 32 * kEpiWarps);
      int all = 1;
#pragma unroll
      for (int w = 0; w < kEpiWarps; ++w) all &= ctrl->vote[i & 1][w];
      if (!all) break;
      tc_fence_after();
      const GradUnit g = grad_unit(p, share.unit(i));
      const int row = g.mt * 2 * BM + static_cast<int>(rank) * BM + q * 32 + lane;
      const bool valid = row < (g.dw ? p.V : p.T);
      const int n0 = g.nt * kBN + cg * (kBN / 2);
      const int chunks = valid ? min(4, (p.D - n0 + 31) / 32) : 0;  // D is a multiple of 64
      const size_t at = static_cast<size_t>(valid ? row : 0) * p.D + n0;
      const uint32_t acc = lane_addr + static_cast<uint32_t>(b * kBN);
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t te = smem_u32(&ctrl->tempty[b]);
          if (rank == 0) mbar_arrive(&ctrl->tempty[b]);
          else mbar_arrive_cluster(mapa_shared(te, 0));
        }
      };
      if (g.dw && p.accumulate) {
        for_tmem_chunks<4>(acc, 0, [&](const uint32_t(&r)[32], int c) {
          if (c < chunks) add_dw<FP32>(p, at + c * 32, r, scale);
        }, release);
      } else if (g.dw) {
        // 128 bytes of each row at a time through shared memory, stored as whole lines
        // (straight from the registers, 32 bytes a lane: the backward of 256 tokens 82 us
        // for 74 in bf16, 113 for 105 in fp32)
        const int all_chunks = min(4, (p.D - n0 + 31) / 32);  // of the tile, valid rows or not
        for_tmem_chunks<4>(acc, 0, [&](const uint32_t(&r)[32], int c) {
          if (c >= all_chunks) return;  // the same for the group
          const int h = FP32 ? 0 : c & 1;
          if (h == 0) {
            if (leader) bulk_wait_read<0>();  // the store before has read the buffer
            named_bar_sync(bar, 128);
          }
#pragma unroll
          for (int v = 0; v < (FP32 ? 8 : 4); ++v) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = FP32 ? __float_as_uint(__uint_as_float(r[(4 * v + e) & 31]) * scale)
                          : pack_bf16x2(__uint_as_float(r[(8 * v + 2 * e) & 31]) * scale,
                                        __uint_as_float(r[(8 * v + 2 * e + 1) & 31]) * scale);
            const uint32_t ci = static_cast<uint32_t>(h * 4 + v);
            st_shared_v4(rowbase + ((ci ^ r7) << 4), w[0], w[1], w[2], w[3]);
          }
          if (FP32 || h == 1) {  // D is a multiple of 64
            fence_proxy_async_smem();
            named_bar_sync(bar, 128);
            if (leader) {
              // (the map counts two bytes)
              tma_store_2d(&p.tmDw, buf, (n0 + (c - h) * 32) * (FP32 ? 2 : 1),
                           g.mt * 2 * BM + static_cast<int>(rank) * BM);
              bulk_commit();
            }
          }
        }, release);
      } else if (p.slices > 1) {
        float* dst = p.part + static_cast<size_t>(g.slice) * p.T * p.D + at;
        for_tmem_chunks<4>(acc, 0, [&](const uint32_t(&r)[32], int c) {
          if (c >= chunks) return;
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            const uint32_t w[8] = {r[k],     r[k + 1], r[k + 2], r[k + 3],
                                   r[k + 4], r[k + 5], r[k + 6], r[k + 7]};
            st_global_v8(dst + c * 32 + k, w);
          }
        }, release);
      } else {
        const float f = valid && p.rowfac ? __ldg(p.rowfac + row) : 1.f;
        for_tmem_chunks<4>(acc, 0, [&](const uint32_t(&r)[32], int c) {
          if (c >= chunks) return;
          uint4* dst = reinterpret_cast<uint4*>(p.dH + at + c * 32);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(r[8 * k + 2 * e]) * f,
                                 __uint_as_float(r[8 * k + 2 * e + 1]) * f);
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }, release);
      }
      if (++b == 2) {
        b = 0;
        aph ^= 1u;
      }
    }
    if (leader) bulk_wait<0>();
    __syncwarp();
  }
  __syncthreads();
  cluster_sync_all();  // the leader's MMAs are drained before either CTA frees TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kBN);
  }
}

// dH = rowfac times the slices' sums, in their order; eight columns a thread.
__global__ void __launch_bounds__(256) k_join_dh(const float* __restrict__ part, int slices,
                                                 int64_t n8, int D8,
                                                 const float* __restrict__ rowfac,
                                                 uint16_t* __restrict__ dH, int* status) {
  pdl_enter();
  if (read_status(status) != 0) return;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n8) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 8
  for (int s = 0; s < slices; ++s) {
    const float4* src = reinterpret_cast<const float4*>(part) + (s * n8 + i) * 2;
    const float4 x = __ldcs(src), y = __ldcs(src + 1);
    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
  }
  const float f = rowfac ? __ldg(rowfac + i / D8) : 1.f;
  reinterpret_cast<uint4*>(dH)[i] =
      make_uint4(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f),
                 pack_bf16x2(b.x * f, b.y * f), pack_bf16x2(b.z * f, b.w * f));
}

// The slices of dH's K: as many as make its tiles' slices about half the pairs, at least
// kLeastKb k-blocks each. Those pairs then read W and G at the MMAs' rate while the
// others write dW, and both end together (backward of V 50304, D 768, in us: T 256, 3
// tiles, in 8, 12, 16, 24 slices 77, 72, 76, 81; T 1024, 12 tiles, in 1, 3, 6 slices
// 306, 167, 183; T 4096, 48 tiles, in 1, 2 slices 612, 630).
constexpr int kLeastKb = 8, kMostSlices = 36, kMostSliceUnits = 54;

int dh_slices(int64_t T, int64_t V, int64_t D, int pairs) {
  const int64_t tiles = cdiv(T, 2 * BM) * cdiv(D, kBN);
  const int64_t half = std::min(pairs, 76) * 36 / 76;
  return static_cast<int>(
      std::max<int64_t>(1, std::min((2 * half + tiles) / (2 * tiles), cdiv(V, BK) / kLeastKb)));
}

}  // namespace

size_t logprob_part_bytes(int64_t T, int64_t D) {
  return static_cast<size_t>(std::min<int64_t>(4 * kMostSlices * T * D,
                                               4 * int64_t(kMostSliceUnits) * 2 * BM * kBN));
}

cudaError_t launch_logprob_grads(const LogprobArgs& p, const uint16_t* G, int64_t ldG,
                                 const uint16_t* Hs, const float* rowfac, const float* scale,
                                 float* part, uint16_t* dH, void* dW, int dw_fp32, int accumulate,
                                 cudaStream_t s) {
  GradArgs a = {};
  if (!map_kmajor(&a.tmGk, G, p.T, p.V, ldG) || !map_mnmajor(&a.tmW, p.W, p.V, p.D, p.D) ||
      !map_mnmajor(&a.tmGm, G, p.T, p.V, ldG) || !map_mnmajor(&a.tmHs, Hs, p.T, p.D, p.D))
    return cudaErrorInvalidValue;
  const uint64_t words = static_cast<uint64_t>(p.D) * (dw_fp32 ? 2 : 1);
  if (!make_bf16_map(&a.tmDw, dW, words, p.V, words * 2, 64, BM)) return cudaErrorInvalidValue;
  const int most = p.num_sms / 2;
  a.n_nt = tiles_of(p.D, kBN);
  a.m_dh = tiles_of(p.T, 2 * BM);
  a.n_dw = tiles_of(p.V, 2 * BM) * a.n_nt;
  a.slices = dh_slices(p.T, p.V, p.D, most);
  a.kb_dw = tiles_of(p.T, BK);
  a.kb_dh = tiles_of(p.V, BK);
  const int n_dh = a.m_dh * a.n_nt * a.slices;
  a.T = p.T, a.V = p.V, a.D = p.D;
  a.dH = dH, a.part = part, a.rowfac = rowfac;
  a.dW = dW, a.scale = scale, a.accumulate = accumulate;
  a.status = p.status;
  a.deal = deal_units(a.n_dw, a.kb_dw, n_dh, cdiv(a.kb_dh, a.slices));
  const dim3 grid(static_cast<unsigned>(2 * std::min(a.n_dw + n_dh, most))), block(kThreads);
  const cudaError_t e =
      dw_fp32 ? launch_pdl(k_logprob_grads<true>, grid, block, L::TOTAL, s, a)
              : launch_pdl(k_logprob_grads<false>, grid, block, L::TOTAL, s, a);
  if (e != cudaSuccess || a.slices == 1) return e;
  const int64_t n8 = static_cast<int64_t>(p.T) * p.D / 8;
  return launch_pdl(k_join_dh, dim3(static_cast<unsigned>((n8 + 255) / 256)), dim3(256), 0, s,
                    static_cast<const float*>(part), a.slices, n8, p.D / 8, rowfac, dH, p.status);
}

}  // namespace ss
