// ss_logprob_fwd.cu -- the softmax partials of the head's log-probabilities over
// the whole vocabulary: logits S = H W^T tile by tile (M = T, N = V, K = D) on CTA
// pairs, of which only a scaled sum of exponentials per row and 128 columns leaves
// the chip.
//
// A log-probability is the difference of two numbers near 10, so the logits want
// more than the tensor core's accumulator gives: it truncates after every 16
// products, and the loss grows with the sum's size and length (the log-sum-exp of
// logits of standard deviation 3 comes out 6e-6 too small at D 768 and 1.7e-5 at
// D 2048, the same way for every token, where fp32 sums rounded to nearest are
// 1e-6 off either way). So K is cut into runs of kRunKb k-blocks, each in a TMEM
// accumulator of its own; the epilogue warps add the runs in registers, rounded to
// nearest, 128 columns of a row per thread: 2.9e-6 too small, whatever D.
//
// The chosen ids' logits are taken from those registers too: what truncation is
// left then falls on both terms of the difference alike for tokens drawn from the model
// (1.3e-6 off either way, with no shift); for ids that are not, whose logits are smaller,
// the log-sum-exp's shift stays (ids drawn uniformly: logp 2.7e-6 too large at V 50257,
// D 1088, where plain fp32 products are 1.1e-6 off either way). And no row of W is read
// again (16384 tokens of 64 ids: gathered rows took 228 us). k_bin_ids sorts the
// ids of each 32 tokens by the 128 columns they fall into; a warp, which holds those
// columns of those tokens, looks up the few that are its own.
//
// T 16384, V 50304, D 768: 712 us, 1.78 PFLOP/s; T 8192, D 2048: 907 us, 1.86. The
// tensor pipe is active in 74% of the cycles (T 4096, 1.90 GHz); the rest is the
// runs' ends, where the MMAs wait for an accumulator.
//
// The protocol is that of ss_gemm2.cuh (pairs of CTAs on 256 x 256 tiles, warp 0
// TMA producer, warp 1 MMA issuer, eight epilogue warps, bounded waits); the two
// accumulators alternate between runs instead of tiles. A tile's exponentials run
// beside the next tile's first runs, as its sums are in registers by then.
#include <algorithm>
#include <limits>

#include "ss_gemm.cuh"
#include "ss_gemm2.cuh"
#include "ss_logprob.cuh"

namespace ss {

namespace {

// k-blocks of 64 in one accumulator (T 16384, V 50304, D 768: 753, 722 and 687 us for
// 4, 6 and 12)
constexpr int kRunKb = 6;
constexpr int kIdRows = 32;  // tokens whose ids are sorted together: an epilogue warp's
constexpr int kBN = kBnLogits;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kHalf = kBN / 2;  // columns of a row per epilogue thread
static_assert(kHalf == 128, "seven bits of a sorted id");
constexpr int kMostBins = SS_MAX_V / kHalf;
constexpr double kLog2eExact = 1.4426950408889634074;
// the exponent of a sum that is infinite: a number, so that differences of it are too
constexpr float kMostExponent = std::numeric_limits<float>::max();
// From this exponent on, what rounding it leaves of the largest logit is no less than what
// fp32 leaves of the log-sum-exp, and can be hundreds: the logit itself is subtracted.
constexpr float kFar = 0x1p24f;
using L = Gemm2Smem<kBN, kStages, 0>;

struct FwdArgs {
  int T, V, m_tiles, n_tiles, k_blocks, group_m;
  HeadCap head;
  float2* part;  // [2 n_tiles][T]: (n, s), 2^n s
  int K;
  const uint32_t* sorted;    // [groups][32 K]: column in its bin, row and k of each id
  const uint16_t* bin_ends;  // [groups][2 n_tiles]: where each bin's ids end
  float* z;                  // [groups][32 K]: the sorted ids' logits
  int* status;
};

// The ids of 32 tokens by column bin, as column | row << 7 | k << 12, and where each bin
// ends. The order within a bin is any: each id's logit goes its way back by row and k. A
// block per 32 tokens.
__global__ void __launch_bounds__(256) k_bin_ids(const int32_t* __restrict__ ids, int K, int T,
                                                 int V, int bins, uint32_t* __restrict__ sorted,
                                                 uint16_t* __restrict__ bin_ends, int* status) {
  __shared__ int count[kMostBins];
  __shared__ int s_warp[8];
  __shared__ int s_go;
  pdl_enter();
  if (threadIdx.x == 0) s_go = read_status(status) == 0;
  for (int i = threadIdx.x; i < bins; i += 256) count[i] = 0;
  __syncthreads();
  if (!s_go) return;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kIdRows;
  const int n = (T - t0 < kIdRows ? static_cast<int>(T - t0) : kIdRows) * K;
  const int32_t* mine = ids + t0 * K;
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int id = __ldg(mine + i);
    bad |= id < -1 || id >= V;
    if (id >= 0 && id < V) atomicAdd(&count[id / kHalf], 1);
  }
  if (bad) set_status(status, SS_ERR_TARGET_RANGE);
  __syncthreads();
  // exclusive sums: consecutive bins per thread, then over the warps
  const int per = (bins + 255) / 256, b0 = threadIdx.x * per;
  int sum = 0;
  for (int b = b0; b < min(b0 + per, bins); ++b) sum += count[b];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int at = upto - sum;
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  uint16_t* ends = bin_ends + static_cast<int64_t>(blockIdx.x) * bins;
  for (int b = b0; b < min(b0 + per, bins); ++b) {
    const int c = count[b];
    count[b] = at;
    at += c;
    ends[b] = static_cast<uint16_t>(at);
  }
  __syncthreads();
  uint32_t* out = sorted + t0 * K;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int id = __ldg(mine + i);
    if (id < 0 || id >= V) continue;
    out[atomicAdd(&count[id / kHalf], 1)] =
        static_cast<uint32_t>(id % kHalf) | static_cast<uint32_t>(i / K) << 7 |
        static_cast<uint32_t>(i % K) << 12;
  }
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// tcgen05.wait::ld that names the registers it waits for
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// acc[k] (+)= the 128 columns from `taddr` on, two to a word
template <bool FIRST>
__device__ __forceinline__ void take_run(uint32_t taddr, uint64_t (&acc)[kHalf / 2]) {
  uint32_t ra[16], rb[16];
  auto add = [&](const uint32_t(&r)[16], int c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint64_t v = f32x2_bits(r[2 * k], r[2 * k + 1]);
      acc[c * 8 + k] = FIRST ? v : add_f32x2(acc[c * 8 + k], v);
    }
  };
  tmem_ld16(taddr, ra);
#pragma unroll
  for (int c = 0; c < kHalf / 16; c += 2) {
    tmem_wait16(ra);
    tmem_ld16(taddr + (c + 1) * 16, rb);
    add(ra, c);
    tmem_wait16(rb);
    if (c + 2 < kHalf / 16) tmem_ld16(taddr + (c + 2) * 16, ra);
    add(rb, c + 1);
  }
}

// acc[i] for an i that the warp agrees on, as registers have no index: branches down to
// one of eight, then selections (branches alone: 16384 tokens of 64 ids 18 us more)
template <int LO, int N>
__device__ __forceinline__ uint64_t pick(const uint64_t (&acc)[kHalf / 2], int i) {
  if constexpr (N == 8) {
    const uint64_t a = (i & 1) ? acc[LO + 1] : acc[LO], b = (i & 1) ? acc[LO + 3] : acc[LO + 2];
    const uint64_t c = (i & 1) ? acc[LO + 5] : acc[LO + 4], d = (i & 1) ? acc[LO + 7] : acc[LO + 6];
    const uint64_t e = (i & 2) ? b : a, f = (i & 2) ? d : c;
    return (i & 4) ? f : e;
  } else {
    return i < LO + N / 2 ? pick<LO, N / 2>(acc, i) : pick<LO + N / 2, N / 2>(acc, i);
  }
}

template <bool CAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_logprob_forward(const __grid_constant__ CUtensorMap tmH,
                      const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ FwdArgs p) {
  pdl_enter();
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_go;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  GemmCtrl* ctrl = reinterpret_cast<GemmCtrl*>(smem + L::CTRL_OFFSET);
  const uint32_t tiles = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

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
    tma_prefetch_map(&tmH);
    tma_prefetch_map(&tmW);
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
  const GemmShape shp{p.m_tiles, p.n_tiles, p.k_blocks, 0, 0, nullptr, p.group_m};
  const int num_units = p.m_tiles * p.n_tiles;

  if (warp == 0) {
    // ------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_ph = 0;
      bool ok = true;
      // W is re-read by every row tile, H by every column tile: both stay in L2
      const bool again = p.m_tiles > 1;
      const uint64_t keep = l2_evict_last();
      for (int u = pair; ok && u < num_units; u += npairs) {
        int mt, nt;
        unit_tile(shp, u, mt, nt);
        const int m0 = mt * 2 * BM + static_cast<int>(rank) * BM;
        const int n0 = nt * kBN + static_cast<int>(rank) * kHalf;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(&ctrl->empty[s], ph ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = smem_u32(&ctrl->full[s]);
          if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * L::STAGE_BYTES);
          const uint32_t fb = rank == 0 ? fb_local : mapa_shared(fb_local, 0);
          const uint32_t dst = tiles + s * L::STAGE_BYTES;
          tma_load_2d_pair(dst, &tmH, fb, kb * BK, m0);
          if (again) tma_load_2d_pair_hint(dst + L::A_BYTES, &tmW, fb, kb * BK, n0, keep);
          else tma_load_2d_pair(dst + L::A_BYTES, &tmW, fb, kb * BK, n0);
          issued |= 1u << s;
          issued_ph = (issued_ph & ~(1u << s)) | (ph << s);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
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
      constexpr uint32_t idesc = idesc_bf16_f32(2 * BM, kBN, false, false);
      int s = 0, b = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int u = pair; ok && u < num_units; u += npairs) {
        for (int k0 = 0; ok && k0 < p.k_blocks; k0 += kRunKb) {
          if (!mbar_wait(&ctrl->tempty[b], aph ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * kBN);
          const int k1 = min(k0 + kRunKb, p.k_blocks);
          for (int kb = k0; kb < k1; ++kb) {
            if (!mbar_wait(&ctrl->full[s], ph, abort_flag, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_addr = tiles + s * L::STAGE_BYTES;
            const uint32_t b_addr = a_addr + L::A_BYTES;
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k)
              mma_bf16_pair(d_tmem, sdesc_sw128(a_addr + k * 32, 16, 1024),
                            sdesc_sw128(b_addr + k * 32, 16, 1024), idesc,
                            (kb > k0 || k > 0) ? 1u : 0u);
            mma_commit_pair(&ctrl->empty[s], 0x3);
            if (++s == kStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (!ok) break;
          mma_commit_pair(&ctrl->tfull[b], 0x3);
          if (++b == 2) {
            b = 0;
            aph ^= 1u;
          }
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
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + cg * kHalf;
    const int runs = (p.k_blocks + kRunKb - 1) / kRunKb;
    int b = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int u = pair; ok && u < num_units; u += npairs) {
      int mt, nt;
      unit_tile(shp, u, mt, nt);
      const int t0 = (mt * 2 + static_cast<int>(rank)) * BM + q * 32;
      // this warp's ids, asked for ahead of their use behind the runs
      int id0 = 0, id1 = 0;
      uint32_t mine = 0u;  // lane l: the l-th
      const uint32_t* sorted = p.sorted + static_cast<int64_t>(t0) * p.K;
      if (t0 < p.T) {
        const int bin = nt * 2 + cg;
        const uint16_t* ends = p.bin_ends + static_cast<int64_t>(t0 / kIdRows) * (2 * p.n_tiles);
        id0 = bin ? __ldg(ends + bin - 1) : 0;
        id1 = __ldg(ends + bin);
      }
      uint64_t acc[kHalf / 2];
      for (int run = 0; run < runs; ++run) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctrl->tfull[b], aph, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = lane_addr + static_cast<uint32_t>(b * kBN);
        if (run == 0) take_run<true>(at, acc);
        else take_run<false>(at, acc);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t te = smem_u32(&ctrl->tempty[b]);
          if (rank == 0) mbar_arrive(&ctrl->tempty[b]);
          else mbar_arrive_cluster(mapa_shared(te, 0));
        }
        if (++b == 2) {
          b = 0;
          aph ^= 1u;
        }
        if (run == 0 && id0 + lane < id1) mine = __ldg(sorted + id0 + lane);
      }
      if (!ok) break;
      const int t = t0 + lane;
      const int nv = p.V - (nt * kBN + cg * kHalf);  // valid columns, the same for the warp
      float m = -INFINITY, s = 0.f;
      if (nv > 0) {
        if constexpr (CAP) {
          // z = cap / (1 + exp(-s / tau)), two logits to an operation where there is one
          // (with the known largest value below: 745 us instead of 764 at T 16384, D 768)
          const uint64_t nk1 = f32x2(-p.head.k1, -p.head.k1), one = f32x2(1.f, 1.f);
          const uint64_t cap = f32x2(p.head.cap, p.head.cap);
#pragma unroll
          for (int k = 0; k < kHalf / 2; ++k) {
            float x, y;
            f32x2_split(mul_f32x2(acc[k], nk1), x, y);
            f32x2_split(add_f32x2(f32x2(ex2_approx(x), ex2_approx(y)), one), x, y);
            acc[k] = mul_f32x2(f32x2(rcp_approx(x), rcp_approx(y)), cap);
          }
        }
        if (nv < kHalf) {  // the vocabulary ends inside
#pragma unroll
          for (int k = 0; k < kHalf / 2; ++k) {
            float x, y;
            f32x2_split(acc[k], x, y);
            acc[k] = f32x2(2 * k < nv ? x : -INFINITY, 2 * k + 1 < nv ? y : -INFINITY);
          }
        }
        // 32 ids at a time: the row's lane has the logit, the id's lane keeps it, so
        // that they are stored in a row (an id's own place in [T, K] straight from the
        // row's lane: 45 us more for 16384 tokens of 64)
        for (int i = id0; i < id1; i += 32) {
          const int n = min(32, id1 - i);
          if (i > id0 && lane < n) mine = __ldg(sorted + i + lane);
          float kept = 0.f;
          for (int l = 0; l < n; ++l) {
            const uint32_t e = __shfl_sync(0xffffffffu, mine, l);
            float x, y;
            f32x2_split(pick<0, kHalf / 2>(acc, static_cast<int>(e & 127u) / 2), x, y);
            x = __shfl_sync(0xffffffffu, (e & 1u) ? y : x, static_cast<int>((e >> 7) & 31u));
            if (lane == l) kept = x;
          }
          if (lane < n) p.z[static_cast<int64_t>(t0) * p.K + i + lane] = kept;
        }
        bool far = false;
        if (CAP && p.head.cap <= kStoredCapMax) {
          // no logit is above it, and exp(-cap) is a normal number
          m = rintf(p.head.cap * kLog2e);
        } else {
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int k = 0; k < kHalf / 2; ++k) {
            float x, y;
            f32x2_split(acc[k], x, y);
            m0 = fmaxf(m0, x);
            m1 = fmaxf(m1, y);
          }
          const float top = fmaxf(m0, m1);
          m = rintf(top * kLog2e);
          far = fabsf(m) >= kFar && fabsf(top) < INFINITY;
          if (__any_sync(0xffffffffu, far)) {
            const uint64_t off = far ? f32x2(-top, -top) : f32x2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kHalf / 2; ++k) acc[k] = add_f32x2(acc[k], off);
          }
        }
        // a row of -infinity alone, or of NaN, and one with an infinity have no number to
        // subtract; the sum of the latter is infinite, or a NaN
        const float r2 = fabsf(m) < INFINITY && !far ? m : 0.f;
        const uint64_t k2 = f32x2(kLog2e, kLog2e), nr2 = f32x2(-r2, -r2);
        uint64_t s0 = f32x2(0.f, 0.f), s1 = s0;
#pragma unroll
        for (int k = 0; k < kHalf / 2; k += 2) {
          float x0, y0, x1, y1;
          f32x2_split(fma_f32x2(acc[k], k2, nr2), x0, y0);
          f32x2_split(fma_f32x2(acc[k + 1], k2, nr2), x1, y1);
          s0 = add_f32x2(s0, f32x2(ex2_approx(x0), ex2_approx(y0)));
          s1 = add_f32x2(s1, f32x2(ex2_approx(x1), ex2_approx(y1)));
        }
        float a0, a1, a2, a3;
        f32x2_split(s0, a0, a1);
        f32x2_split(s1, a2, a3);
        s = (a0 + a1) + (a2 + a3);
        // What shifts every token's sum the same way, and so adds up over a sequence:
        // kLog2e is 1.93e-8 below log2(e), so that exp(z) came out as exp(z (1 - 1.3e-8))
        // (1.2e-7 less where z is 9), which is put back at the mean of z log2(e). That mean
        // is the logarithm of the sum less the entropy of the 128 columns in bits, which is
        // taken as 3.6, what logits of standard deviation 3 have; it is 0 to 7, and the
        // difference worth 3.4e-8 at most. And the hardware's exponential is 5.0e-8 too
        // small on average (a million points). Log-probabilities of tokens drawn from the
        // model are then off by 1e-8 on average, 9e-7 with neither this nor integers as
        // the exponents (a cap of 30).
        constexpr float kUnder = static_cast<float>((kLog2eExact - double(kLog2e)) /
                                                    (kLog2eExact * kLog2eExact));
        const float mean = fmaxf(r2 + __log2f(s) - 3.6f, -1e6f);  // (s can be 0)
        s = fmaf(s, fmaf(kUnder, mean, 5.0e-8f), s);
      }
      if (t < p.T)
        p.part[static_cast<size_t>(nt * 2 + cg) * p.T + t] = make_float2(fminf(m, kMostExponent), s);
    }
  }
  __syncthreads();
  cluster_sync_all();  // the leader's MMAs are drained before either CTA frees TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kBN);
  }
}

// --------------------------------------------------------------- few tokens
//
// One token or two (a served model's next position): W is read once, at memory's rate,
// and the products run on the fp32 pipe beside it, where a tile of 256 tokens on the
// tensor cores would be mostly empty (V 50304, D 768, one token: 16.7 us with the merge,
// 77 MB, where the tiles take 35; four tokens: 29 and 31, D 2048 64 and 58). A warp
// takes kRows vocabulary rows at a time, each lane eight columns of every 256; the
// tokens lie in shared memory. The ids' logits are more rows of the same kind, so that
// the sums are the same ones.
constexpr int kFewThreads = 256, kRows = 4;

struct FewArgs {
  const uint16_t *H, *W;
  const int32_t* ids;
  int T, V, D, K;
  float cap, tau;
  float2* part;  // [gridDim.x][T]
  float* z;      // [T, K]
  int* status;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// acc[r][t] = W[row[r]] . H[t], in every lane
template <int N, int R>
__device__ __forceinline__ void rows_dot(const FewArgs& p, const uint4* h, const uint4* (&row)[R],
                                         int lane, float (&acc)[R][N]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < N; ++t) acc[r][t] = 0.f;
  const int d8 = p.D / 8;
#pragma unroll 3
  for (int c = lane; c < d8; c += 32) {
    uint4 w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = __ldcs(row[r] + c);
    float x[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) unpack8(w[r], x[r]);
#pragma unroll
    for (int t = 0; t < N; ++t) {
      float y[8];
      unpack8(h[t * d8 + c], y);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r][t] = fmaf(x[r][i], y[i], acc[r][t]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < N; ++t) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
}

// (m, s) and the logit z
__device__ __forceinline__ void take_logit(float z, float& m, float& s) {
  if (z == -INFINITY) return;  // adds nothing, and leaves no number to subtract if it is first
  const float top = fmaxf(m, z);
  // (the first logit: exp(-inf) = 0; a NaN stays in the sum; an infinity makes it infinite)
  s = fabsf(top) < INFINITY ? s * expf(m - top) + expf(z - top) : s + z;
  m = top;
}
__device__ __forceinline__ void take_partial(float om, float os, float& m, float& s) {
  if (om == -INFINITY && os == 0.f) return;
  const float top = fmaxf(m, om);
  s = top < INFINITY ? s * expf(m - top) + os * expf(om - top) : s + os;
  m = top;
}

template <int N>
__global__ void __launch_bounds__(kFewThreads) k_logprob_few(const FewArgs p) {
  pdl_enter();
  extern __shared__ uint4 s_h[];
  __shared__ float2 s_part[kFewThreads / 32][N];
  __shared__ int s_go;
  if (threadIdx.x == 0) s_go = read_status(p.status) == 0;
  const int d8 = p.D / 8;
  for (int i = threadIdx.x; i < N * d8; i += kFewThreads)
    s_h[i] = i < p.T * d8 ? __ldg(reinterpret_cast<const uint4*>(p.H) + i)
                          : make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  if (!s_go) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int w = static_cast<int>(blockIdx.x) * (kFewThreads / 32) + warp;
  const int warps = static_cast<int>(gridDim.x) * (kFewThreads / 32);
  const uint4* W = reinterpret_cast<const uint4*>(p.W);
  auto capped = [&](float z) { return p.cap > 0.f ? p.cap / (1.f + expf(-z / p.tau)) : z; };
  // the chosen ids, one at a time
  for (int64_t i = w; i < static_cast<int64_t>(p.T) * p.K; i += warps) {
    const int id = __ldg(p.ids + i);
    if (id < 0 || id >= p.V) {
      if (lane == 0 && id != -1) set_status(p.status, SS_ERR_TARGET_RANGE);
      continue;
    }
    const uint4* row[1] = {W + static_cast<int64_t>(id) * d8};
    float acc[1][1];
    rows_dot<1, 1>(p, s_h + (i / p.K) * d8, row, lane, acc);
    if (lane == 0) p.z[i] = capped(acc[0][0]);
  }
  // lane t keeps token t's running pair
  float m = -INFINITY, s = 0.f;
  for (int v0 = w * kRows; v0 < p.V; v0 += warps * kRows) {
    const uint4* row[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      row[r] = W + static_cast<int64_t>(min(v0 + r, p.V - 1)) * d8;
    float acc[kRows][N];
    rows_dot<N, kRows>(p, s_h, row, lane, acc);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float z = acc[r][0];
#pragma unroll
      for (int t = 1; t < N; ++t)
        if (lane == t) z = acc[r][t];
      if (lane < N && v0 + r < p.V) take_logit(capped(z), m, s);
    }
  }
  if (lane < N) s_part[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x < p.T) {
    for (int k = 1; k < kFewThreads / 32; ++k)
      take_partial(s_part[k][threadIdx.x].x, s_part[k][threadIdx.x].y, m, s);
    // 2^n s, log2(e) in two parts
    constexpr float kLog2eLo = static_cast<float>(kLog2eExact - double(kLog2e));
    const float n = fminf(rintf(m * kLog2e), kMostExponent);
    if (fabsf(n) < kFar) s *= exp2f(fmaf(m, kLog2eLo, fmaf(m, kLog2e, -n)));
    p.part[static_cast<int64_t>(blockIdx.x) * p.T + threadIdx.x] = make_float2(n, s);
  }
}

template <int N>
cudaError_t few(const FewArgs& p, int blocks, cudaStream_t s) {
  return launch_pdl(k_logprob_few<N>, dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads),
                    static_cast<size_t>(N) * p.D * 2, s, p);
}

// Units walk groups of this many rows column tile by column tile, so that W is
// read from memory once per group.
constexpr int kGroupRows = 8192;

}  // namespace

int logprob_few_parts(int64_t T, int64_t V, int num_sms) {
  if (T > kFewTokens) return 0;
  const int64_t want = (V + kRows * kFewThreads / 32 - 1) / (kRows * kFewThreads / 32);
  return static_cast<int>(std::min<int64_t>({want, int64_t(num_sms) * 3, kMostFewParts}));
}

cudaError_t launch_logprob_few(const LogprobArgs& p, int K, const int32_t* ids, int parts,
                               float2* part, float* z, cudaStream_t s) {
  const FewArgs a{p.H, p.W, ids, p.T, p.V, p.D, K, p.cap, p.tau, part, z, p.status};
  static_assert(kFewTokens == 2 && 2 * SS_MAX_D * 2 <= 64 * 1024, "tokens in shared memory");
  return p.T <= 1 ? few<1>(a, parts, s) : few<2>(a, parts, s);
}

cudaError_t launch_bin_ids(const LogprobArgs& p, const int32_t* ids, int K, int bins,
                           uint32_t* sorted, uint16_t* bin_ends, cudaStream_t s) {
  return launch_pdl(k_bin_ids, dim3(static_cast<unsigned>((p.T + kIdRows - 1) / kIdRows)),
                    dim3(256), 0, s, ids, K, p.T, p.V, bins, sorted, bin_ends, p.status);
}

cudaError_t launch_logprob_partials(const LogprobArgs& p, int K, const uint32_t* sorted,
                                    const uint16_t* bin_ends, float2* part, float* z,
                                    cudaStream_t s) {
  CUtensorMap tH, tW;
  const uint64_t row = static_cast<uint64_t>(p.D) * 2;
  if (!make_bf16_map(&tH, p.H, p.D, p.T, row, BK, BM) ||
      !make_bf16_map(&tW, p.W, p.D, p.V, row, BK, kHalf))
    return cudaErrorInvalidValue;
  const FwdArgs a{p.T,      p.V, (p.T + 2 * BM - 1) / (2 * BM), (p.V + kBN - 1) / kBN, p.D / BK,
                  kGroupRows / (2 * BM), p.head, part, K, sorted, bin_ends, z, p.status};
  const int pairs = std::min(a.m_tiles * a.n_tiles, p.num_sms / 2);
  const dim3 grid(static_cast<unsigned>(2 * pairs)), block(kThreads);
  return p.cap > 0.f ? launch_pdl(k_logprob_forward<true>, grid, block, L::TOTAL, s, tH, tW, a)
                     : launch_pdl(k_logprob_forward<false>, grid, block, L::TOTAL, s, tH, tW, a);
}

}  // namespace ss
