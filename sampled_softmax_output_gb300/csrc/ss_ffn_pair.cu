// ss_ffn_pair.cu -- the feed-forward block's products on CTA pairs: one 2-SM
// tcgen05.mma.cta_group::2 per 256 x 256 x 16 step, the protocol of
// ss_gemm2.cuh over a list of jobs.
//
// A job is one product with up to two segments of K (dX = dG Wg + dU Wu is one
// accumulation over 2 F), its operands' tensor maps and majors, and its tiles.
// A launch runs one or more jobs; pair p runs the units p, p + pairs, ... of
// all jobs' tiles in a row, or those that ss_ffn_plan.h deals it (dX and dW).
//
// gate/up: the two CTAs of a pair hold the two halves of the MMA's N, and here
// the leader's half is 128 rows of Wg and the peer's 128 rows of Wu. Columns
// 0-127 of each accumulator row are then G and 128-255 U of the same features,
// so the epilogue has both in one thread and the activation and product need
// no exchange.
//
// What bounds it: the MMAs of a k-block of 256 x 256 x 64 take 512 cycles from
// resident operands; with TMA feeding them 575 to 580 (K of 4096 and more), and
// what an epilogue moves through shared memory or to global memory comes on top,
// about 9 cycles a KB. So outputs are stored from registers, 32 bytes a lane,
// wherever rows lie on 32-byte boundaries (gate/up with G, U and A kept: 784 ->
// 675 cycles a k-block at D 768, 745 with their low bits); else (gate/up, dA) through shared memory by
// TMA, since half sectors cost more than that (T 3001, D 1352, F 3640: 56 us
// against 68). In a steady loop the board's power does: it draws 1380 W at 1.55
// to 1.75 GHz.
//   one launch at a time      gate/up       down          dA            dX and dW
//   T 65536, D 768, F 2048    285 us 1.45   154 us 1.34   240 us 0.86   555 us 1.86 PFLOP/s
//   T 8192, D 2048, F 5504    226    1.64   129    1.43   165    1.12   507    1.82
// (As a training step calls them: low bits of G and U written and read, dropout and
// residual in the down projection; launch, exit and the last, partly filled round of
// tiles included. The low bits are 20 and 28 us of the first and third column at
// T 65536, 7 and 6 us at T 8192.)
//
// Roles per CTA: warp 0 TMA producer, warp 1 MMA issuer (the leader's), warps
// 2-9 epilogue: two column groups of four warps, one accumulator row per
// thread, two TMEM accumulators so that the epilogue of a tile runs beside the
// MMAs of the next.
#include <algorithm>
#include <type_traits>

#include "ss_ffn.cuh"
#include "ss_gemm.cuh"
#include "ss_gemm2.cuh"

namespace ss {

namespace {

// kUp, kGradAct: outputs staged in shared memory; ...Wide: stored from registers
enum Kind { kUp, kUpWide, kDown, kGradAct, kGradActWide, kGrads };

constexpr int kBN = 256, kNarrowBN = 192;
template <int KIND>
constexpr bool kIsUp = KIND == kUp || KIND == kUpWide;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxJobs = 4;

struct PairJob {
  CUtensorMap a[2], b[2];  // per segment of K (gate/up: b per CTA of the pair)
  int kb[2];               // k-blocks of each segment
  int a_mn, b_mn;          // 1: MN-major operand
  int m_tiles, n_tiles;
  int units_end;  // units of this job and of those before it
};

// The output of a job of kGrads: rows x cols of bf16 or fp32, times scale.
struct GradOut {
  void* out;
  int rows, cols;
  float scale;
  int fp32, accumulate;
  int wide;  // rows on 32-byte boundaries
};

// Staging of 32-column chunks: 128 rows x 64 bytes, 64-byte swizzle (16-byte
// chunk c of row r at c ^ ((r >> 1) & 3)), so that eight rows' 16-byte accesses
// to the same chunk hit all 32 banks.
constexpr uint32_t kChunkBytes = 128 * 64;
__device__ __forceinline__ uint32_t chunk_addr(uint32_t buf, int row, int c) {
  return buf + static_cast<uint32_t>(row) * 64u +
         static_cast<uint32_t>((c ^ ((row >> 1) & 3)) * 16);
}

// Up to 32 columns (nv of them, a multiple of 8) of one row of bf16: whole
// sectors where the rows are 32-byte aligned.
__device__ __forceinline__ void store_row32(uint16_t* dst, const uint32_t (&w)[16], int nv,
                                            bool wide) {
  if (wide) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (c * 16 >= nv) break;
      const uint32_t x[8] = {w[8 * c],     w[8 * c + 1], w[8 * c + 2], w[8 * c + 3],
                             w[8 * c + 4], w[8 * c + 5], w[8 * c + 6], w[8 * c + 7]};
      st_global_v8(dst + c * 16, x);
    }
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v * 8 < nv)
        reinterpret_cast<uint4*>(dst)[v] =
            make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
  }
}

// The low bits of the elements j .. j + 3 of a chunk; og, ou: packed bf16 pairs,
// o the index of the first
template <int N>
__device__ __forceinline__ uint32_t low_of(const uint32_t (&rg)[32], const uint32_t (&ru)[32],
                                           const uint32_t (&og)[N], const uint32_t (&ou)[N], int j,
                                           int o) {
  const float g[4] = {__uint_as_float(rg[j]), __uint_as_float(rg[j + 1]),
                      __uint_as_float(rg[j + 2]), __uint_as_float(rg[j + 3])};
  const float u[4] = {__uint_as_float(ru[j]), __uint_as_float(ru[j + 1]),
                      __uint_as_float(ru[j + 2]), __uint_as_float(ru[j + 3])};
  return low_bits4(g, u, og[o], og[o + 1], ou[o], ou[o + 1]);
}

template <int KIND>
struct PairCfg;
template <>
struct PairCfg<kUp> {
  static constexpr int kStages = 5, kBufs = 1, kTensors = 3;  // G, U, A chunks
};
template <>
struct PairCfg<kUpWide> {
  static constexpr int kStages = 6, kBufs = 0, kTensors = 0;
};
template <>
struct PairCfg<kGradActWide> {
  static constexpr int kStages = 5, kBufs = 2, kTensors = 2;  // G, U in
};
template <>
struct PairCfg<kDown> {
  static constexpr int kStages = 6, kBufs = 0, kTensors = 0;
};
template <>
struct PairCfg<kGradAct> {
  static constexpr int kStages = 4, kBufs = 3, kTensors = 2;  // G, U in; dG, dU out, in place
};
template <>
struct PairCfg<kGrads> {
  static constexpr int kStages = 6, kBufs = 0, kTensors = 0;
};

template <int KIND>
constexpr int epi_bytes() {
  return 2 * PairCfg<KIND>::kBufs * PairCfg<KIND>::kTensors * static_cast<int>(kChunkBytes);
}

template <int KIND>
struct PairArgs {
  PairJob job[KIND == kGrads ? kMaxJobs : 1];
  int n_jobs, group_m;
  int T, D, F, act;
  int ldo;  // elements between the rows of G, U, A (gate/up) or dG, dU (dA)
  uint16_t *G, *U, *A;
  // kUp: G, U, A (stores); kGradAct: G, U (loads), dG, dU (stores)
  CUtensorMap m[4];
  int save;  // gate/up: G and U are kept
  uint8_t* R;  // nullable; rows of ldr bytes
  int ldr;
  // kDown
  const uint16_t* residual;
  uint16_t* Y;
  int wide;  // Y's rows on 32-byte boundaries
  DropArgs drop;
  float scale;  // kGradAct, kGradActWide
  GradOut grad[KIND == kGrads ? kMaxJobs : 1];
  int* status;
  UnitDeal deal;  // kGrads
};

// The units of one pair, one after the other: p, p + pairs, ..., or (kGrads) as
// they are dealt.
template <int KIND>
struct UnitWalk {
  int at, end, step;
  __device__ __forceinline__ UnitWalk(const PairArgs<KIND>& p, int pair, int npairs)
      : at(pair), end(p.job[0].units_end), step(npairs) {}
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ void next() { at += step; }
  __device__ __forceinline__ int unit() const { return at; }
};
template <>
struct UnitWalk<kGrads> {
  PairShare share;
  int at = 0;
  __device__ __forceinline__ UnitWalk(const PairArgs<kGrads>& p, int pair, int npairs)
      : share(share_of(p.deal, pair, npairs)) {}
  __device__ __forceinline__ bool more() const { return at < share.count(); }
  __device__ __forceinline__ void next() { ++at; }
  __device__ __forceinline__ int unit() const { return share.unit(at); }
};

struct Unit {
  int job, mt, nt;
};
template <int KIND>
__device__ __forceinline__ Unit find_unit(const PairArgs<KIND>& p, int u) {
  int j = 0, first = 0;
  if constexpr (KIND == kGrads) {
    while (j + 1 < p.n_jobs && u >= p.job[j].units_end) first = p.job[j++].units_end;
  }
  GemmShape shp{p.job[j].m_tiles, p.job[j].n_tiles, 0, 0, 0, nullptr, p.group_m};
  Unit r{j, 0, 0};
  unit_tile(shp, u - first, r.mt, r.nt);
  return r;
}

// BN: columns of a tile, 256, or 192 for gate/up and dA
template <int KIND, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_ffn_pair(const __grid_constant__ PairArgs<KIND> p) {
  pdl_enter();
  using C = PairCfg<KIND>;
  constexpr int STAGES = C::kStages;
  using L = Gemm2Smem<kBN, STAGES, epi_bytes<KIND>()>;
  static_assert(sizeof(GemmCtrl) <= L::CTRL_BYTES, "control block");
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_go;
  __shared__ uint64_t s_load[2][4];  // kGradAct: chunk loads per column group and buffer
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  GemmCtrl* ctrl = reinterpret_cast<GemmCtrl*>(smem + L::CTRL_OFFSET);
  const uint32_t tiles = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  int* status = p.status;
  constexpr int n_chunks = BN / 64;  // of 32 columns, to a column group (dA)

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->tempty[b], 2 * kEpiWarps);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&s_load[0][0] + i, 1);
    mbar_init(&ctrl->drain, 1);
    ctrl->abort_flag = 0;
    s_go = read_status(status) == 0;
    fence_mbar_init();
    for (int j = 0; j < p.n_jobs; ++j) {
      tma_prefetch_map(&p.job[j].a[0]);
      tma_prefetch_map(&p.job[j].b[0]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctrl->tmem_base, 2 * kBN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  // Both CTAs take the same decision: an earlier error seen by either ends both.
  const bool go_pair = s_go && ld_shared_cluster_u32(mapa_shared(smem_u32(&s_go), rank ^ 1u));
  const uint32_t tmem_base = ctrl->tmem_base;
  volatile int* abort_flag = &ctrl->abort_flag;

  if (!go_pair) {
    // nothing to do but to meet the peer below
  } else if (warp == 0) {
    // ------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      // A is read by the few column tiles of its rows at about the same time
      // (transposed operands of dW: evict-first took the launch from 708 to 660
      // cycles a k-block); B by every row tile: kept in L2
      const uint64_t stream = l2_evict_first(), keep = l2_evict_last();
      const uint32_t full0 = mapa_shared(smem_u32(&ctrl->full[0]), 0);  // the leader's
      int s = 0;
      uint32_t ph = 0, issued = 0;  // k-blocks issued
      bool ok = true;
      for (UnitWalk<KIND> w(p, pair, npairs); ok && w.more(); w.next()) {
        const Unit un = find_unit(p, w.unit());
        const PairJob& job = p.job[un.job];
        const int m0 = un.mt * 2 * BM + static_cast<int>(rank) * BM;
        // this CTA's half of the tile's N; gate/up: the same 128 features of
        // the CTA's own matrix
        const int n0 = kIsUp<KIND> ? un.nt * (BN / 2)
                                   : un.nt * BN + static_cast<int>(rank) * (BN / 2);
        // one k-loop per form of the operands, chosen once per unit: this thread
        // issues every copy, and branches between them cost 8% of dX and dW
        auto load_unit = [&](auto a_form, auto b_form) {
          constexpr bool A_MN = decltype(a_form)::value, B_MN = decltype(b_form)::value;
          // half a tile's columns: two boxes of 64 (BN 192: the last 32 of them for
          // nothing), or one of BN / 2 rows
          constexpr uint32_t b_bytes = B_MN ? 16384u : BN * BK;
#pragma unroll 1
          for (int seg = 0; ok && seg < 2; ++seg) {
            const CUtensorMap* ma = &job.a[seg];
            const CUtensorMap* mb =
                &job.b[kIsUp<KIND> ? static_cast<int>(rank) : seg];
            const int k_end = job.kb[seg] * BK;
#pragma unroll 1
            for (int k = 0; k < k_end; k += BK) {
              if (!mbar_wait(&ctrl->empty[s], ph ^ 1u, abort_flag, status)) {
                ok = false;
                break;
              }
              if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * (L::A_BYTES + b_bytes));
              const uint32_t fb = full0 + s * 8;
              const uint32_t a_dst = tiles + s * L::STAGE_BYTES;
              const uint32_t b_dst = a_dst + L::A_BYTES;
              if constexpr (A_MN) {
                tma_load_2d_pair_hint(a_dst, ma, fb, m0, k, stream);
                tma_load_2d_pair_hint(a_dst + 8192, ma, fb, m0 + 64, k, stream);
              } else {
                tma_load_2d_pair(a_dst, ma, fb, k, m0);
              }
              if constexpr (B_MN) {
                tma_load_2d_pair_hint(b_dst, mb, fb, n0, k, keep);
                tma_load_2d_pair_hint(b_dst + 8192, mb, fb, n0 + 64, k, keep);
              } else {
                tma_load_2d_pair_hint(b_dst, mb, fb, k, n0, keep);
              }
              ++issued;
              if (++s == STAGES) {
                s = 0;
                ph ^= 1u;
              }
            }
          }
        };
        if constexpr (KIND == kGradAct || KIND == kGradActWide) {
          load_unit(std::false_type{}, std::true_type{});
        } else if constexpr (KIND == kGrads) {
          if (job.a_mn) load_unit(std::true_type{}, std::true_type{});
          else load_unit(std::false_type{}, std::true_type{});
        } else {
          load_unit(std::false_type{}, std::false_type{});
        }
      }
      if (rank == 0) {
        // every copy of both CTAs that the leader armed must land
        for (uint32_t i = issued > STAGES ? issued - STAGES : 0u; i < issued; ++i)
          mbar_drain(&ctrl->full[i % STAGES], (i / STAGES) & 1u, status);
      } else if (!ok) {
        // aborted: give this CTA's copies in flight, which land on the
        // leader's barriers, a bounded moment before shared memory goes
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
      for (UnitWalk<KIND> w(p, pair, npairs); ok && w.more(); w.next()) {
        const Unit un = find_unit(p, w.unit());
        const PairJob& job = p.job[un.job];
        const int kbs = job.kb[0] + job.kb[1];
        const bool a_mn = job.a_mn != 0, b_mn = job.b_mn != 0;
        const uint32_t idesc = a_mn   ? idesc_bf16_f32(2 * BM, BN, true, true)
                               : b_mn ? idesc_bf16_f32(2 * BM, BN, false, true)
                                      : idesc_bf16_f32(2 * BM, BN, false, false);
        if (!mbar_wait(&ctrl->tempty[b], aph ^ 1u, abort_flag, status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * kBN);
        bool ready = false;
        for (int kb = 0; kb < kbs; ++kb) {
          if (!ready && !mbar_wait(&ctrl->full[s], ph, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = tiles + s * L::STAGE_BYTES;
          const uint32_t b_addr = a_addr + L::A_BYTES;
          const int sn = s + 1 == STAGES ? 0 : s + 1;
          const uint32_t pn = sn == 0 ? ph ^ 1u : ph;
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k) {
            const uint64_t ad = a_mn ? sdesc_sw128(a_addr + k * 2048, 8192, 1024)
                                     : sdesc_sw128(a_addr + k * 32, 16, 1024);
            const uint64_t bd = b_mn ? sdesc_sw128(b_addr + k * 2048, 8192, 1024)
                                     : sdesc_sw128(b_addr + k * 32, 16, 1024);
            mma_bf16_pair(d_tmem, ad, bd, idesc, (kb | k) != 0 ? 1u : 0u);
            // the next stage is asked for while this one's MMAs queue (2 to 3%)
            if (k == 1) ready = mbar_try_wait(smem_u32(&ctrl->full[sn]), pn);
          }
          mma_commit_pair(&ctrl->empty[s], 0x3);
          s = sn;
          ph = pn;
        }
        if (!ok) break;
        mma_commit_pair(&ctrl->tfull[b], 0x3);
        if (++b == 2) {
          b = 0;
          aph ^= 1u;
        }
      }
      mma_commit_pair(&ctrl->drain, 0x1);
      mbar_drain(&ctrl->drain, 0, status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;         // TMEM lane quarter this warp may access
    const int cg = (warp - 2) / 4;  // column group
    const int row = q * 32 + lane;
    const bool leader = ((threadIdx.x - 64) & 127) == 0;  // of the column group
    const int bar = 1 + 2 * cg;                           // the group's named barrier
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    // this group's staging
    constexpr uint32_t kBufBytes = C::kTensors * kChunkBytes;
    const uint32_t stage = tiles + L::EPI_OFFSET + static_cast<uint32_t>(cg * C::kBufs) * kBufBytes;
    const uint64_t seed = KIND == kDown ? drop_seed(p.drop) : 0;
    int b = 0;
    uint32_t aph = 0;

    [[maybe_unused]] auto row_of = [&](const Unit& x) {
      return (x.mt * 2 + static_cast<int>(rank)) * BM + row;
    };
    // dA: round r of this group is chunk r % n_chunks of its tile r / n_chunks; the
    // G and U chunks of round r are loaded ahead into buffer r % kBufs. kGradAct:
    // two rounds ahead, replaced there by dG and dU and stored from there;
    // kGradActWide: read into registers, and the buffer is loaded again at once.
    [[maybe_unused]] int round = 0, n_rounds = 0;
    [[maybe_unused]] auto chunk_at = [&](int r, int& col, int& mrow) {
      const int turn = r / n_chunks;
      const Unit un = find_unit(p, pair + turn * npairs);
      col = un.nt * BN + cg * (BN / 2) + (r - turn * n_chunks) * 32;
      mrow = (un.mt * 2 + static_cast<int>(rank)) * BM;
    };
    [[maybe_unused]] auto load_round = [&](int r) {  // by the group's leader
      int col, mrow;
      chunk_at(r, col, mrow);
      const int buf = r % C::kBufs;
      uint64_t* bar_ld = &s_load[cg][buf];
      mbar_arrive_expect_tx(bar_ld, 2 * kChunkBytes);
      const uint32_t dst = stage + static_cast<uint32_t>(buf) * kBufBytes;
      tma_load_2d(dst, &p.m[0], bar_ld, col, mrow);
      tma_load_2d(dst + kChunkBytes, &p.m[1], bar_ld, col, mrow);
    };
    if constexpr (KIND == kGradAct || KIND == kGradActWide) {
      constexpr int kAhead = KIND == kGradAct ? 2 : C::kBufs;
      const int num_units = p.job[0].units_end;
      const int my_units = pair < num_units ? (num_units - pair + npairs - 1) / npairs : 0;
      n_rounds = my_units * n_chunks;
      if (leader)
        for (int r = 0; r < min(kAhead, n_rounds); ++r) load_round(r);
    }

    // dA: the low bits of the next chunk's G and U, loaded one chunk ahead
    [[maybe_unused]] uint32_t low_next[8] = {};
    [[maybe_unused]] auto load_low = [&](const Unit& x, int i) {
      const int tt = row_of(x), f = x.nt * BN + cg * (BN / 2) + i * 32;
      if (p.R && tt < p.T && f < p.F)
        ld_global_v8(p.R + static_cast<size_t>(tt) * p.ldr + f, low_next);
    };
    [[maybe_unused]] auto take_low = [&](uint32_t (&low)[8], const Unit& x, UnitWalk<KIND> w,
                                         int i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) low[k] = low_next[k];
      if (i + 1 < n_chunks) {
        load_low(x, i + 1);
      } else {
        w.next();
        if (w.more()) load_low(find_unit(p, w.unit()), 0);
      }
    };
    if constexpr (KIND == kGradAct || KIND == kGradActWide) {
      UnitWalk<KIND> w(p, pair, npairs);
      if (w.more()) load_low(find_unit(p, w.unit()), 0);
    }
    int turn = 0;
    for (UnitWalk<KIND> w(p, pair, npairs); w.more(); w.next(), ++turn) {
      const bool ok = mbar_wait(&ctrl->tfull[b], aph, abort_flag, status);
      bool go = __all_sync(0xffffffffu, ok);
      if constexpr (C::kBufs > 0) {  // the epilogue's warps meet at barriers: agree first
        if (lane == 0) ctrl->vote[turn & 1][warp - 2] = go ? 1 : 0;
        group_sync(2, 32 * kEpiWarps);
        const int* v = ctrl->vote[turn & 1];
        int all = 1;
#pragma unroll
        for (int i = 0; i < kEpiWarps; ++i) all &= v[i];
        go = all != 0;
      }
      if (!go) break;
      tc_fence_after();
      const Unit un = find_unit(p, w.unit());
      const int mrow = (un.mt * 2 + static_cast<int>(rank)) * BM;  // first row of this CTA
      const int t = mrow + row;
      const uint32_t acc = lane_addr + static_cast<uint32_t>(b * kBN);
      // hands the accumulator back once it is in registers
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(&ctrl->tempty[b]);
          else mbar_arrive_cluster(mapa_shared(smem_u32(&ctrl->tempty[b]), 0));
        }
      };

      // body(r, i) over the 32-column chunks of this group. What moves TMEM wants
      // the warp whole; the rows and columns that a body leaves out part it.
      [[maybe_unused]] auto for_chunks = [&](auto&& body) {
        for_tmem_chunks<4>(
            acc, cg * 4,
            [&](const uint32_t(&r)[32], int i) {
              body(r, i);
              __syncwarp();
            },
            release);
      };

      if constexpr (KIND == kUpWide) {
        const bool valid = t < p.T;
        dispatch_act(p.act, [&](auto act) {
          constexpr int ACT = decltype(act)::value;
#pragma unroll 1
          for (int c0 = cg * 32; c0 < BN / 2; c0 += 64) {  // within the tile's features
            const int f0 = un.nt * (BN / 2) + c0;
            uint32_t rg[32], ru[32];
            __syncwarp();
            tmem_ld32(acc + c0, rg);
            tmem_ld32(acc + BN / 2 + c0, ru);
            tmem_ld_wait(rg);
            tmem_ld_wait(ru);
            if (c0 + 64 >= BN / 2) release();
            const size_t at = static_cast<size_t>(valid ? t : 0) * p.ldo + f0;
            const int nv = valid ? min(32, p.F - f0) : 0;
            uint32_t low[8] = {};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (c * 16 >= nv) break;
              uint32_t oa[8], og[8], ou[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int j = c * 16 + 2 * k;
                const float g0 = __uint_as_float(rg[j]), g1 = __uint_as_float(rg[j + 1]);
                const float u0 = __uint_as_float(ru[j]), u1 = __uint_as_float(ru[j + 1]);
                float a0, a1, unused;
                act_eval<ACT, false>(g0, a0, unused);
                act_eval<ACT, false>(g1, a1, unused);
                oa[k] = pack_bf16x2(a0 * u0, a1 * u1);
                og[k] = pack_bf16x2(g0, g1);
                ou[k] = pack_bf16x2(u0, u1);
              }
              st_global_v8(p.A + at + c * 16, oa);
              if (p.save) {
                st_global_v8(p.G + at + c * 16, og);
                st_global_v8(p.U + at + c * 16, ou);
              }
              if (p.R) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  low[c * 4 + k] = low_of(rg, ru, og, ou, c * 16 + 4 * k, 2 * k);
              }
            }
            if (p.R && nv > 0) st_global_v8(p.R + static_cast<size_t>(t) * p.ldr + f0, low);
          }
        });
      } else if constexpr (KIND == kGradActWide) {
        const bool valid = t < p.T;
        dispatch_act_low(p.act, p.R != nullptr, [&](auto act, auto with_low) {
          constexpr int ACT = decltype(act)::value;
          constexpr bool LOW = decltype(with_low)::value;
#pragma unroll 1
          for (int i = 0; i < n_chunks; ++i, ++round) {
            const int c0 = cg * (BN / 2) + i * 32;
            const int f0 = un.nt * BN + c0;
            const int buf = round % C::kBufs;
            const uint32_t sg = stage + static_cast<uint32_t>(buf) * kBufBytes;
            [[maybe_unused]] uint32_t low[8];
            if constexpr (LOW) take_low(low, un, w, i);
            uint32_t r[32];
            __syncwarp();
            tmem_ld32(acc + c0, r);
            mbar_wait(&s_load[cg][buf], (round / C::kBufs) & 1, abort_flag, status);
            __syncwarp();
            uint32_t g[16], v[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t at = chunk_addr(sg, row, c);
              uint32_t x[4];
              ld_shared_v4(at, x);
              g[4 * c] = x[0], g[4 * c + 1] = x[1], g[4 * c + 2] = x[2], g[4 * c + 3] = x[3];
              ld_shared_v4(at + kChunkBytes, x);
              v[4 * c] = x[0], v[4 * c + 1] = x[1], v[4 * c + 2] = x[2], v[4 * c + 3] = x[3];
            }
            tmem_ld_wait(r);
            if (i + 1 == n_chunks) release();
            // The group has read the buffer. Without the fence a read may still be on
            // its way behind the MMAs' own when the next copy lands.
            fence_proxy_async_smem();
            group_sync(bar, 128);
            if (leader && round + C::kBufs < n_rounds) load_round(round + C::kBufs);
            const int nv = valid ? min(32, p.F - f0) : 0;
            if (nv > 0) {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float o[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float dA = __uint_as_float(r[2 * k + h]) * p.scale;
                  const int e = 2 * k + h;
                  float gv = h ? bf16_hi(g[k]) : bf16_lo(g[k]);
                  float uv = h ? bf16_hi(v[k]) : bf16_lo(v[k]);
                  if constexpr (LOW) {
                    gv = refine(g[k], halves_g(low[e >> 2]), e & 3);
                    uv = refine(v[k], halves_u(low[e >> 2]), e & 3);
                  }
                  float a, d;
                  act_eval<ACT, true>(gv, a, d);
                  o[h] = dA * uv * d;
                  o[2 + h] = dA * a;
                }
                g[k] = pack_bf16x2(o[0], o[1]);
                v[k] = pack_bf16x2(o[2], o[3]);
              }
              const size_t at = static_cast<size_t>(t) * p.ldo + f0;
              store_row32(p.G + at, g, nv, true);
              store_row32(p.U + at, v, nv, true);
            }
          }
        });
      } else if constexpr (KIND == kUp) {
        dispatch_act(p.act, [&](auto act) {
          constexpr int ACT = decltype(act)::value;
#pragma unroll 1
          for (int c0 = cg * 32; c0 < BN / 2; c0 += 64) {  // within the tile's features
            const int f0 = un.nt * (BN / 2) + c0;
            uint32_t rg[32], ru[32];
            __syncwarp();
            tmem_ld32(acc + c0, rg);
            tmem_ld32(acc + BN / 2 + c0, ru);
            tmem_ld_wait(rg);
            tmem_ld_wait(ru);
            if (c0 + 64 >= BN / 2) release();
            // the last store from the staging buffer has read it
            if (leader) bulk_wait_read<0>();
            group_sync(bar, 128);
            uint32_t low[8] = {};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t ga[4], gg[4], gu[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int at = c * 8 + 2 * k;
                const float g0 = __uint_as_float(rg[at]), g1 = __uint_as_float(rg[at + 1]);
                const float u0 = __uint_as_float(ru[at]), u1 = __uint_as_float(ru[at + 1]);
                float a0, a1, unused;
                act_eval<ACT, false>(g0, a0, unused);
                act_eval<ACT, false>(g1, a1, unused);
                ga[k] = pack_bf16x2(a0 * u0, a1 * u1);
                gg[k] = pack_bf16x2(g0, g1);
                gu[k] = pack_bf16x2(u0, u1);
              }
              const uint32_t at = chunk_addr(stage, row, c);
              st_shared_v4(at, ga[0], ga[1], ga[2], ga[3]);
              if (p.save) {
                st_shared_v4(at + kChunkBytes, gg[0], gg[1], gg[2], gg[3]);
                st_shared_v4(at + 2 * kChunkBytes, gu[0], gu[1], gu[2], gu[3]);
              }
              if (p.R) {
                low[2 * c] = low_of(rg, ru, gg, gu, c * 8, 0);
                low[2 * c + 1] = low_of(rg, ru, gg, gu, c * 8 + 4, 2);
              }
            }
            if (p.R && t < p.T && f0 < p.F)
              st_global_v8(p.R + static_cast<size_t>(t) * p.ldr + f0, low);
            fence_proxy_async_smem();
            group_sync(bar, 128);
            if (leader) {
              if (f0 < p.F && mrow < p.T) {
                tma_store_2d(&p.m[2], stage, f0, mrow);
                if (p.save) {
                  tma_store_2d(&p.m[0], stage + kChunkBytes, f0, mrow);
                  tma_store_2d(&p.m[1], stage + 2 * kChunkBytes, f0, mrow);
                }
              }
              bulk_commit();
            }
          }
        });
      } else if constexpr (KIND == kGradAct) {
        dispatch_act_low(p.act, p.R != nullptr, [&](auto act, auto with_low) {
          constexpr int ACT = decltype(act)::value;
          constexpr bool LOW = decltype(with_low)::value;
#pragma unroll 1
          for (int i = 0; i < n_chunks; ++i, ++round) {
            const int c0 = cg * (BN / 2) + i * 32;
            const int f0 = un.nt * BN + c0;
            const int buf = round % 3;
            const uint32_t sg = stage + static_cast<uint32_t>(buf) * kBufBytes;
            [[maybe_unused]] uint32_t low[8];
            if constexpr (LOW) take_low(low, un, w, i);
            uint32_t r[32];
            __syncwarp();
            tmem_ld32(acc + c0, r);
            mbar_wait(&s_load[cg][buf], (round / 3) & 1, abort_flag, status);
            __syncwarp();
            tmem_ld_wait(r);
            if (i + 1 == n_chunks) release();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t at = chunk_addr(sg, row, c);
              uint32_t wg[4], wu[4];
              ld_shared_v4(at, wg);
              ld_shared_v4(at + kChunkBytes, wu);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float o[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float dA = __uint_as_float(r[c * 8 + 2 * k + h]) * p.scale;
                  const int e = c * 8 + 2 * k + h;
                  float g = h ? bf16_hi(wg[k]) : bf16_lo(wg[k]);
                  float uu = h ? bf16_hi(wu[k]) : bf16_lo(wu[k]);
                  if constexpr (LOW) {
                    g = refine(wg[k], halves_g(low[e >> 2]), e & 3);
                    uu = refine(wu[k], halves_u(low[e >> 2]), e & 3);
                  }
                  float a, d;
                  act_eval<ACT, true>(g, a, d);
                  o[h] = dA * uu * d;
                  o[2 + h] = dA * a;
                }
                wg[k] = pack_bf16x2(o[0], o[1]);
                wu[k] = pack_bf16x2(o[2], o[3]);
              }
              st_shared_v4(at, wg[0], wg[1], wg[2], wg[3]);
              st_shared_v4(at + kChunkBytes, wu[0], wu[1], wu[2], wu[3]);
            }
            fence_proxy_async_smem();
            group_sync(bar, 128);
            if (leader) {
              if (f0 < p.F && mrow < p.T) {
                tma_store_2d(&p.m[2], sg, f0, mrow);
                tma_store_2d(&p.m[3], sg + kChunkBytes, f0, mrow);
              }
              bulk_commit();
              if (round + 2 < n_rounds) {
                bulk_wait_read<1>();  // the store of round - 1, from buffer (round + 2) % 3
                load_round(round + 2);
              }
            }
          }
        });
      } else if constexpr (KIND == kDown) {
        const bool valid = t < p.T;
        const int n0 = un.nt * kBN + cg * 128;
        const int ncols = valid ? min(128, p.D - n0) : 0;
        const size_t base = static_cast<size_t>(valid ? t : 0) * p.D + n0;
        // the residual of the next chunk, loaded one chunk ahead
        uint32_t rn[16];
        auto load_residual = [&](int i) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (p.residual && i * 32 + v * 8 < ncols)
              x = *reinterpret_cast<const uint4*>(p.residual + base + i * 32 + v * 8);
            rn[4 * v] = x.x, rn[4 * v + 1] = x.y, rn[4 * v + 2] = x.z, rn[4 * v + 3] = x.w;
          }
        };
        load_residual(0);
        for_chunks([&](const uint32_t(&r)[32], int i) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = rn[k];
          if (i < 3) load_residual(i + 1);
          const int nv = min(32, ncols - i * 32);
          if (nv <= 0) return;
          const size_t at = base + i * 32;
          uint32_t kept = 0xffffffffu;  // bit k: column k stays
          if (p.drop.mode == kDropAll) kept = 0u;
          if (p.drop.mode == kDropRandom) {
            kept = 0u;
            auto keep = [&](int k, bool yes) { kept |= (yes ? 1u : 0u) << k; };
            const uint64_t e = p.drop.offset + at;
            if (e & 1) for_kept<32, true>(seed, e, p.drop.thr, keep);
            else for_kept<32, false>(seed, e, p.drop.thr, keep);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float lo = bf16_lo(w[k]), hi = bf16_hi(w[k]);
            if ((kept >> (2 * k)) & 1u) lo = fmaf(__uint_as_float(r[2 * k]), p.drop.scale, lo);
            if ((kept >> (2 * k + 1)) & 1u)
              hi = fmaf(__uint_as_float(r[2 * k + 1]), p.drop.scale, hi);
            w[k] = pack_bf16x2(lo, hi);
          }
          store_row32(p.Y + at, w, nv, p.wide);
        });
      } else {
        const GradOut& go_ = p.grad[un.job];
        const bool valid = t < go_.rows;
        const int n0 = un.nt * kBN + cg * 128;
        const int ncols = min(128, go_.cols - n0);
        const size_t base = static_cast<size_t>(valid ? t : 0) * go_.cols + n0;
        const float scale = go_.scale;
        if (ncols <= 0) release();
        else if (go_.fp32)
          for_chunks([&](const uint32_t(&r)[32], int i) {
            const int nv = min(32, ncols - i * 32);
            if (nv <= 0 || !valid) return;
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(go_.out) + base + i * 32);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k * 4 >= nv) break;
              float4 o = make_float4(
                  __uint_as_float(r[4 * k]) * scale, __uint_as_float(r[4 * k + 1]) * scale,
                  __uint_as_float(r[4 * k + 2]) * scale, __uint_as_float(r[4 * k + 3]) * scale);
              if (go_.accumulate) {
                const float4 old = dst[k];
                o.x += old.x, o.y += old.y, o.z += old.z, o.w += old.w;
              }
              dst[k] = o;
            }
          });
        else
          for_chunks([&](const uint32_t(&r)[32], int i) {
            const int nv = min(32, ncols - i * 32);
            if (nv <= 0 || !valid) return;
            uint16_t* dst = static_cast<uint16_t*>(go_.out) + base + i * 32;
            uint32_t w[16] = {};
            if (go_.accumulate) {
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (v * 8 < nv) {
                  const uint4 x = reinterpret_cast<const uint4*>(dst)[v];
                  w[4 * v] = x.x, w[4 * v + 1] = x.y, w[4 * v + 2] = x.z, w[4 * v + 3] = x.w;
                }
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              w[k] = pack_bf16x2(fmaf(__uint_as_float(r[2 * k]), scale, bf16_lo(w[k])),
                                 fmaf(__uint_as_float(r[2 * k + 1]), scale, bf16_hi(w[k])));
            store_row32(dst, w, nv, go_.wide);
          });
      }
      if (++b == 2) {
        b = 0;
        aph ^= 1u;
      }
    }
    if constexpr (KIND == kGradAct || KIND == kGradActWide) {
      // aborted: the chunk loads in flight land before shared memory goes
      constexpr int kAhead = KIND == kGradAct ? 2 : C::kBufs;
      if (leader && round < n_rounds)
        for (int r = round; r < min(round + kAhead, n_rounds); ++r)
          mbar_drain(&s_load[cg][r % C::kBufs], (r / C::kBufs) & 1, status);
    }
    if constexpr (KIND == kUp || KIND == kGradAct) {
      if (leader) bulk_wait<0>();
    }
    __syncwarp();
  }
  __syncthreads();
  cluster_sync_all();  // the leader's MMAs are drained before either CTA frees TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kBN);
  }
}

// ------------------------------------------------------------- host side

// From this K on the MMAs, not the eight bytes of G, U, dG and dU for each
// element of dA, bound that product: 256 x 256 elements move 512 KB, as long as
// about 17 k-blocks. kGradActWide leaves more shared-memory bandwidth to the
// MMAs (T 16384, D 1024, F 4096: 129 us against 135); kGradAct keeps more
// copies in flight (T 65536, D 768, F 2048: 205 us against 225; both sides without
// the low bits).
constexpr int kActWideKb = 16;

// The units walk groups of this many row tiles column by column: a round of
// the 76 pairs then reads about as many row tiles of A as column tiles of B.
constexpr int kGroupM = 8;

// rows of `cols` bf16 values at each of these on 32-byte boundaries
bool rows_on_sectors(int64_t cols, std::initializer_list<const void*> ps) {
  return cols % 16 == 0 && std::all_of(ps.begin(), ps.end(), [](const void* p) {
           return reinterpret_cast<uintptr_t>(p) % 32 == 0;
         });
}

bool map_chunk(CUtensorMap* m, const uint16_t* p, int64_t rows, int64_t cols, int64_t ld) {
  return make_bf16_map(m, p, cols, rows, ld * 2, 32, 128);
}

template <int KIND, int BN = kBN>
cudaError_t launch_pair(PairArgs<KIND>& p, int num_sms, cudaStream_t s) {
  int end = 0;
  for (int j = 0; j < p.n_jobs; ++j) {
    end += p.job[j].m_tiles * p.job[j].n_tiles;
    p.job[j].units_end = end;
  }
  p.group_m = kGroupM;
  const int pairs = end < num_sms / 2 ? end : num_sms / 2;
  if constexpr (KIND == kGrads) {
    // the three dW, then dX; or only either
    const int n_a = p.n_jobs == kMaxJobs ? p.job[2].units_end : end;
    auto kb = [&](int j) { return p.job[j].kb[0] + p.job[j].kb[1]; };
    p.deal = deal_units(n_a, kb(0), end - n_a, kb(p.n_jobs - 1));
  }
  constexpr int smem = Gemm2Smem<kBN, PairCfg<KIND>::kStages, epi_bytes<KIND>()>::TOTAL;
  return launch_pdl(k_ffn_pair<KIND, BN>, dim3(2 * pairs), dim3(kThreads), smem, s, p);
}

template <int KIND, int BN>
cudaError_t gate_up(const FfnForward& f, cudaStream_t s) {
  PairArgs<KIND> p = {};
  PairJob& j = p.job[0];
  const bool save = f.G != nullptr;
  if (!map_kmajor(&j.a[0], f.X, f.T, f.D, f.D) || !map_kmajor(&j.b[0], f.Wg, f.F, f.D, f.D, BN / 2) ||
      !map_kmajor(&j.b[1], f.Wu, f.F, f.D, f.D, BN / 2))
    return cudaErrorInvalidValue;
  if (KIND == kUp &&
      (!map_chunk(&p.m[2], f.A, f.T, f.F, f.ldo) ||
       (save && (!map_chunk(&p.m[0], f.G, f.T, f.F, f.ldo) || !map_chunk(&p.m[1], f.U, f.T, f.F, f.ldo)))))
    return cudaErrorInvalidValue;
  j.kb[0] = tiles_of(f.D, BK);
  j.m_tiles = tiles_of(f.T, 2 * BM);
  j.n_tiles = tiles_of(f.F, BN / 2);
  p.n_jobs = 1;
  p.T = f.T, p.D = f.D, p.F = f.F, p.act = f.act, p.save = save;
  p.ldo = f.ldo, p.G = f.G, p.U = f.U, p.A = f.A;
  p.R = f.R, p.ldr = f.ldr;
  p.status = f.status;
  return launch_pair<KIND, BN>(p, f.num_sms, s);
}

template <int KIND, int BN>
cudaError_t grad_act(const FfnBackward& f, cudaStream_t s) {
  PairArgs<KIND> p = {};
  PairJob& j = p.job[0];
  if (!map_kmajor(&j.a[0], f.dZ, f.T, f.D, f.D) || !map_mnmajor(&j.b[0], f.Wd, f.D, f.F, f.F))
    return cudaErrorInvalidValue;
  j.b_mn = 1;
  if ((!map_chunk(&p.m[0], f.G, f.T, f.F, f.F) || !map_chunk(&p.m[1], f.U, f.T, f.F, f.F) ||
       !map_chunk(&p.m[2], f.dG, f.T, f.F, f.ldg) || !map_chunk(&p.m[3], f.dU, f.T, f.F, f.ldg)))
    return cudaErrorInvalidValue;
  j.kb[0] = tiles_of(f.D, BK);
  j.m_tiles = tiles_of(f.T, 2 * BM);
  j.n_tiles = tiles_of(f.F, BN);
  p.n_jobs = 1;
  p.T = f.T, p.D = f.D, p.F = f.F, p.act = f.act, p.scale = f.scale;
  p.ldo = f.ldg, p.G = f.dG, p.U = f.dU;
  p.R = const_cast<uint8_t*>(f.R), p.ldr = f.ldr;
  p.status = f.status;
  return launch_pair<KIND, BN>(p, f.num_sms, s);
}

}  // namespace

cudaError_t pair_gate_up(const FfnForward& f, int bn, cudaStream_t s) {
  if (rows_on_sectors(f.ldo, {f.G, f.U, f.A}))
    return bn == kBN ? gate_up<kUpWide, kBN>(f, s) : gate_up<kUpWide, kNarrowBN>(f, s);
  return bn == kBN ? gate_up<kUp, kBN>(f, s) : gate_up<kUp, kNarrowBN>(f, s);
}

cudaError_t pair_grad_act(const FfnBackward& f, int bn, cudaStream_t s) {
  if (tiles_of(f.D, BK) >= kActWideKb && rows_on_sectors(f.ldg, {f.dG, f.dU}))
    return bn == kBN ? grad_act<kGradActWide, kBN>(f, s) : grad_act<kGradActWide, kNarrowBN>(f, s);
  return bn == kBN ? grad_act<kGradAct, kBN>(f, s) : grad_act<kGradAct, kNarrowBN>(f, s);
}

cudaError_t pair_down(const FfnForward& f, cudaStream_t s) {
  PairArgs<kDown> p = {};
  PairJob& j = p.job[0];
  if (!map_kmajor(&j.a[0], f.A, f.T, f.F, f.ldo) || !map_kmajor(&j.b[0], f.Wd, f.D, f.F, f.F))
    return cudaErrorInvalidValue;
  j.kb[0] = tiles_of(f.F, BK);
  j.m_tiles = tiles_of(f.T, 2 * BM);
  j.n_tiles = tiles_of(f.D, kBN);
  p.n_jobs = 1;
  p.T = f.T, p.D = f.D, p.F = f.F;
  p.residual = f.residual, p.Y = f.Y, p.drop = f.drop;
  p.wide = rows_on_sectors(f.D, {f.Y});
  p.status = f.status;
  return launch_pair(p, f.num_sms, s);
}

cudaError_t pair_grads(const FfnBackward& f, int which, cudaStream_t s) {
  PairArgs<kGrads> p = {};
  const int64_t T = f.T, D = f.D, F = f.F;
  if (which & kDoW) {  // dWg, dWu = dG^T X, dU^T X; dWd = dZ^T A: K = T
    const uint16_t* a[3] = {f.dG, f.dU, f.dZ};
    const uint16_t* b[3] = {f.X, f.X, f.A};
    const int64_t rows[3] = {F, F, D}, cols[3] = {D, D, F};
    void* out[3] = {f.dWg, f.dWu, f.dWd};
    for (int i = 0; i < 3; ++i) {
      PairJob& j = p.job[p.n_jobs];
      if (!map_mnmajor(&j.a[0], a[i], T, rows[i], i == 2 ? D : f.ldg) ||
          !map_mnmajor(&j.b[0], b[i], T, cols[i], cols[i]))
        return cudaErrorInvalidValue;
      j.kb[0] = tiles_of(T, BK);
      j.a_mn = j.b_mn = 1;
      j.m_tiles = tiles_of(rows[i], 2 * BM);
      j.n_tiles = tiles_of(cols[i], kBN);
      p.grad[p.n_jobs++] = GradOut{out[i], static_cast<int>(rows[i]), static_cast<int>(cols[i]),
                                   i == 2 ? f.scale : 1.f, f.dw_fp32, f.accumulate,
                                   rows_on_sectors(cols[i], {out[i]})};
    }
  }
  if (which & kDoX) {  // dX = dG Wg + dU Wu: K = F twice
    PairJob& j = p.job[p.n_jobs];
    if (!map_kmajor(&j.a[0], f.dG, T, F, f.ldg) || !map_kmajor(&j.a[1], f.dU, T, F, f.ldg) ||
        !map_mnmajor(&j.b[0], f.Wg, F, D, D) || !map_mnmajor(&j.b[1], f.Wu, F, D, D))
      return cudaErrorInvalidValue;
    j.b_mn = 1;
    j.kb[0] = j.kb[1] = tiles_of(F, BK);
    j.m_tiles = tiles_of(T, 2 * BM);
    j.n_tiles = tiles_of(D, kBN);
    p.grad[p.n_jobs++] = GradOut{f.dX, f.T, f.D, 1.f, 0, 0, rows_on_sectors(D, {f.dX})};
  }
  p.T = f.T, p.D = f.D, p.F = f.F;
  p.status = f.status;
  return launch_pair(p, f.num_sms, s);
}

}  // namespace ss

