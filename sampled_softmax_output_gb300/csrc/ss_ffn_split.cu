// ss_ffn_split.cu -- the feed-forward block's products with K split over a
// thread-block cluster: 128 x BN tiles on single CTAs, the S CTAs of a cluster
// each summing a S-th of K, joined through distributed shared memory.
//
// Out[n, m] = sum_k B[n, k] A[m, k] with the output's contiguous dimension on
// the MMA's M (128 rows of weights) and the tokens on its N (16 to 128). One
// token thus costs a 16-wide MMA next to the weights' bytes, which bound the
// decoding forms: every weight is read once, by TMA, and all SMs stream (T 16,
// D 4096, F 12288: 302 MB in 53 us, 5.7 TB/s; tiles of 56 to 128 rows, so that
// the CTAs number the SMs exactly, took as long).
// Small batches of training have too few 256 x 256 tiles for 76 CTA pairs;
// here a tile is an eighth of that and K gives up to eight CTAs more.
//
// A CTA: warp 0 TMA producer, warp 1 MMA issuer, then all eight warps move the
// accumulator (one TMEM lane = one feature) to shared memory as P[n][m]. After
// a cluster barrier, CTA r sums the columns n = r BN / S ... of all S partial
// tiles in the order of their ranks (no atomics: the same result every time)
// and runs the epilogue on them with four features a lane, so that global
// accesses are contiguous.
#include <algorithm>

#include "ss_ffn.cuh"
#include "ss_gemm.cuh"

namespace ss {

namespace {

enum SplitKind { kSUp, kSDown, kSGradAct, kSGradX, kSGradW };

constexpr int kSplitThreads = 256;
constexpr int kSplitMaxJobs = 3;

// When a kernel of this file waits for the one before it in the stream:
enum SplitWait {
  kWaitFirst,   // before anything
  kWaitLoadA,   // the producer loads A (weights, older than that kernel) before it waits
  kWaitLast,    // reads nothing that kernel writes: before exiting only
};

struct SplitJob {
  CUtensorMap a[2], b[2];  // per segment of K (gate/up: a = Wg, Wu, 64 rows each)
  int kb[2];
  int a_mn, b_mn;
  int m_tiles, n_tiles;
  int tiles_end;  // tiles of this job and of those before it
  // kSGradX, kSGradW: the output, rows x cols with cols on M, times scale
  void* out;
  int rows, cols;
  float scale;
  int fp32, accumulate;
};

template <int KIND>
struct SplitArgs {
  SplitJob job[KIND == kSGradW ? kSplitMaxJobs : 1];
  int n_jobs, wait;
  int T, D, F, act;
  int ldo;  // elements between the rows of G, U, A (gate/up) or dG, dU (dA)
  uint8_t* R;  // nullable: low bits of G and U, rows of ldr bytes
  int ldr;
  const uint16_t *residual, *G_in, *U_in;
  uint16_t *Y, *G, *U, *A;  // kSUp: outputs (G null: not kept); kSGradAct: dG, dU in G, U
  DropArgs drop;
  float scale;
  int* status;
};

template <int BN>
struct SplitSmem {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = BN * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // two CTAs per SM
  static constexpr int STAGES = 110 * 1024 / STAGE_BYTES;
  static constexpr int RING = STAGES * STAGE_BYTES;
  static constexpr int TOTAL = RING + 1024;  // + alignment
  static_assert(BN * BM * 4 <= RING, "the partial tile takes the ring's place");
  static_assert(STAGES >= 3 && STAGES <= 8, "stages");
};

struct SplitCtrl {
  uint64_t full[8], empty[8], done;
  uint32_t tmem_base;
  int abort_flag, go;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

struct F4 {
  float v[4];
};

// P[n][m .. m + 3] at `at`, summed over the partial tiles of a cluster of S
// CTAs, rank by rank, for N places `step` bytes apart whose loads are all
// issued before the first is used.
template <int S, int N>
__device__ __forceinline__ void cluster_sums(uint32_t at, uint32_t step, F4 (&out)[N]) {
  float4 x[N][S];
#pragma unroll
  for (int r = 0; r < S; ++r) {
    const uint32_t base = S == 1 ? at : mapa_shared(at, r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (S == 1) {
        uint32_t w[4];
        ld_shared_v4(base + i * step, w);
        x[i][r] = make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]),
                              __uint_as_float(w[3]));
      } else {
        x[i][r] = ld_cluster_f4(base + i * step);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    out[i] = F4{{x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w}};
#pragma unroll
    for (int r = 1; r < S; ++r) {
      out[i].v[0] += x[i][r].x, out[i].v[1] += x[i][r].y;
      out[i].v[2] += x[i][r].z, out[i].v[3] += x[i][r].w;
    }
  }
}

// fn with the cluster's size as a constant
template <class F>
__device__ __forceinline__ void dispatch_cluster(int S, F&& fn) {
  switch (S) {  // uniform
    case 1: fn(std::integral_constant<int, 1>{}); break;
    case 2: fn(std::integral_constant<int, 2>{}); break;
    case 4: fn(std::integral_constant<int, 4>{}); break;
    default: fn(std::integral_constant<int, 8>{}); break;
  }
}

__device__ __forceinline__ F4 load_bf16x4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return F4{{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)}};
}
__device__ __forceinline__ void store_bf16x4(uint16_t* p, const F4& r) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]));
}

template <int KIND, int BN>
__global__ void __launch_bounds__(kSplitThreads, 2)
    k_ffn_split(const __grid_constant__ SplitArgs<KIND> p, int S) {
  // The next kernel may start once this one has waited itself: it may read
  // before its own wait what kernels older than this one wrote.
  if (p.wait == kWaitFirst) pdl_enter();
  if (p.wait == kWaitLast) pdl_launch_dependents();
  using L = SplitSmem<BN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ SplitCtrl ctrl;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = static_cast<int>(cluster_ctarank());
  constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;

  // this cluster's tile; consecutive clusters share the rows of A
  int tile = static_cast<int>(blockIdx.x) / S, ji = 0;
  if constexpr (KIND == kSGradW) {
    int first = 0;
    while (ji + 1 < p.n_jobs && tile >= p.job[ji].tiles_end) first = p.job[ji++].tiles_end;
    tile -= first;
  }
  const SplitJob& job = p.job[ji];
  const int mt = tile / job.n_tiles, nt = tile % job.n_tiles;
  const int kbs = job.kb[0] + (KIND == kSUp ? 0 : job.kb[1]);
  const int kb0 = static_cast<int>(static_cast<int64_t>(kbs) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(kbs) * (rank + 1) / S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(&ctrl.full[s], 1);
      mbar_init(&ctrl.empty[s], 1);
    }
    mbar_init(&ctrl.done, 1);
    ctrl.abort_flag = 0;
    ctrl.go = read_status(p.status) == 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctrl.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl.tmem_base;
  volatile int* abort_flag = &ctrl.abort_flag;
  // an earlier error: no loads and no outputs, but the cluster's barriers are
  // met (a peer may read this CTA's shared memory)
  const bool go = ctrl.go != 0;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------- producer
    auto load_a = [&](int s, int kb) {
      const uint32_t dst = ring + s * L::STAGE_BYTES;
      if constexpr (KIND == kSUp) {
        tma_load_2d(dst, &job.a[0], &ctrl.full[s], kb * BK, mt * 64);
        tma_load_2d(dst + 8192, &job.a[1], &ctrl.full[s], kb * BK, mt * 64);
      } else {
        const int seg = kb >= job.kb[0] ? 1 : 0;
        const int k = (kb - (seg ? job.kb[0] : 0)) * BK;
        if (job.a_mn) {
          tma_load_2d(dst, &job.a[seg], &ctrl.full[s], mt * BM, k);
          tma_load_2d(dst + 8192, &job.a[seg], &ctrl.full[s], mt * BM + 64, k);
        } else {
          tma_load_2d(dst, &job.a[seg], &ctrl.full[s], k, mt * BM);
        }
      }
    };
    auto load_b = [&](int s, int kb) {
      const uint32_t dst = ring + s * L::STAGE_BYTES + L::A_BYTES;
      const int seg = KIND != kSUp && kb >= job.kb[0] ? 1 : 0;
      const int k = (kb - (seg ? job.kb[0] : 0)) * BK;
      if (BN >= 64 && job.b_mn) {
#pragma unroll
        for (int i = 0; i < BN / 64; ++i)
          tma_load_2d(dst + i * 8192, &job.b[seg], &ctrl.full[s], nt * BN + 64 * i, k);
      } else {
        tma_load_2d(dst, &job.b[seg], &ctrl.full[s], k, nt * BN);
      }
    };
    if (go) {
      const int ahead = min(kb1 - kb0, L::STAGES);  // the ring's first round needs no wait
      for (int i = 0; i < ahead; ++i) {
        mbar_arrive_expect_tx(&ctrl.full[i], L::STAGE_BYTES);
        load_a(i, kb0 + i);
        if (p.wait != kWaitLoadA) load_b(i, kb0 + i);
      }
      if (p.wait == kWaitLoadA) {
        pdl_enter();
        for (int i = 0; i < ahead; ++i) load_b(i, kb0 + i);
      }
      int s = 0;
      uint32_t ph = 0;
      for (int kb = kb0 + ahead; kb < kb1; ++kb) {
        if (!mbar_wait(&ctrl.empty[s], ph, abort_flag, p.status)) break;
        mbar_arrive_expect_tx(&ctrl.full[s], L::STAGE_BYTES);
        load_a(s, kb);
        load_b(s, kb);
        if (++s == L::STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 1 && lane == 0 && go) {
    // -------------------------------------------------------- MMA issuer
    const bool a_mn = KIND != kSUp && job.a_mn, b_mn = BN >= 64 && job.b_mn;
    const uint32_t idesc = a_mn ? (b_mn ? idesc_bf16_f32(BM, BN, true, true)
                                        : idesc_bf16_f32(BM, BN, true, false))
                                : idesc_bf16_f32(BM, BN, false, false);
    int s = 0;
    uint32_t ph = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      // (a failed wait: the MMAs below would read what has not landed; stop)
      if (!mbar_wait(&ctrl.full[s], ph, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t a_addr = ring + s * L::STAGE_BYTES;
      const uint32_t b_addr = a_addr + L::A_BYTES;
#pragma unroll
      for (int k = 0; k < BK / UMMA_K; ++k) {
        const uint64_t ad = a_mn ? sdesc_sw128(a_addr + k * 2048, 8192, 1024)
                                 : sdesc_sw128(a_addr + k * 32, 16, 1024);
        const uint64_t bd = b_mn ? sdesc_sw128(b_addr + k * 2048, 8192, 1024)
                                 : sdesc_sw128(b_addr + k * 32, 16, 1024);
        mma_bf16(tmem, ad, bd, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
      }
      mma_commit(&ctrl.empty[s]);
      if (++s == L::STAGES) {
        s = 0;
        ph ^= 1u;
      }
    }
    mma_commit(&ctrl.done);
  }
  __syncwarp();
  // (kWaitLoadA) `go` is older than the end of the kernel before, which may have
  // recorded an error since: then what it wrote is not to be used. A thread
  // without a role asks, beside the MMAs.
  bool clean = true;
  if (p.wait == kWaitLoadA) {
    pdl_wait();
    if (threadIdx.x == kSplitThreads - 1) clean = read_status(p.status) == 0;
  }

  // ------------------------------------------------- accumulator -> P[n][m]
  // Every block's loads have landed when its MMAs are done, so the ring is free.
  bool ok = go && mbar_wait(&ctrl.done, 0, abort_flag, p.status);
  ok = __syncthreads_and(ok && clean && !*abort_flag) != 0;
  if (ok) {
    tc_fence_after();
    const int q = warp & 3, half = warp >> 2;
    constexpr int kChunks = (BN + 31) / 32;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if ((c & 1) != half) continue;  // uniform in the warp
      uint32_t r[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c * 32, r);
      tmem_ld_wait(r);
      const uint32_t at = ring + static_cast<uint32_t>((c * 32) * BM + q * 32 + lane) * 4u;
#pragma unroll
      for (int n = 0; n < (BN < 32 ? BN : 32); ++n)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + n * BM * 4), "r"(r[n]) : "memory");
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync_all();

  // ------------------------------------------- join the partials, epilogue
  if (ok)
    dispatch_cluster(S, [&](auto cluster) {
      constexpr int CS = decltype(cluster)::value;
      constexpr int n_each = BN / CS;
      const int n_first = rank * n_each;
      const uint64_t seed = KIND == kSDown ? drop_seed(p.drop) : 0;
      // columns a warp takes at a time: two for gate/up (16 lanes each), else one
      constexpr int kStep = KIND == kSUp ? 16 : 8;
      // columns whose partial sums are in flight together in a lane
      constexpr int kMost = KIND == kSUp ? (CS <= 2 ? 4 : 2) : (CS <= 2 ? 8 : CS == 4 ? 4 : 2);
      constexpr int kBatch = n_each / kStep < 1 ? 1 : n_each / kStep < kMost ? n_each / kStep : kMost;
      const int ml = KIND == kSUp ? 4 * (lane & 15) : 4 * lane;
      const int m = mt * (KIND == kSUp ? 64 : BM) + ml;
      const int n_lane = KIND == kSUp ? warp * 2 + (lane >> 4) : warp;
#pragma unroll 1
      for (int n0 = n_lane; n0 < n_each; n0 += kBatch * kStep) {
        const uint32_t at = ring + static_cast<uint32_t>((n_first + n0) * BM + ml) * 4u;
        const int row0 = nt * BN + n_first + n0;
        F4 v[kBatch];
        [[maybe_unused]] F4 w[kBatch];
        [[maybe_unused]] uint2 g_in[kBatch], u_in[kBatch];
        [[maybe_unused]] uint32_t low[kBatch];
        // what else the epilogue reads, all of it on its way before the first use
        // (Y may be the residual: a load after a store would have to wait for it)
        if constexpr (KIND == kSDown) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            w[i] = p.residual && row0 + i * kStep < p.T && m < p.D
                       ? load_bf16x4(p.residual + static_cast<size_t>(row0 + i * kStep) * p.D + m)
                       : F4{{0.f, 0.f, 0.f, 0.f}};
        }
        if constexpr (KIND == kSGradAct) {  // G and U of the same places
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (row0 + i * kStep < p.T && m < p.F) {
              const size_t o = static_cast<size_t>(row0 + i * kStep) * p.F + m;
              u_in[i] = *reinterpret_cast<const uint2*>(p.U_in + o);
              g_in[i] = *reinterpret_cast<const uint2*>(p.G_in + o);
              low[i] = p.R ? *reinterpret_cast<const uint32_t*>(
                                 p.R + static_cast<size_t>(row0 + i * kStep) * p.ldr + m)
                           : 0x88888888u;  // as they are
            }
        }
        [[maybe_unused]] F4 x[kBatch];
        if constexpr (KIND == kSGradAct) {
          cluster_sums<CS>(at, kStep * BM * 4, x);
        } else {
          cluster_sums<CS>(at, kStep * BM * 4, v);
        }
        if constexpr (KIND == kSUp) cluster_sums<CS>(at + 64 * 4, kStep * BM * 4, w);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int row = row0 + i * kStep;
          if constexpr (KIND == kSUp) {
            if (row >= p.T || m >= p.F) continue;
            const size_t o = static_cast<size_t>(row) * p.ldo + m;
            F4 a;
            dispatch_act(p.act, [&](auto act) {
              constexpr int ACT = decltype(act)::value;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float unused;
                act_eval<ACT, false>(v[i].v[k], a.v[k], unused);
                a.v[k] *= w[i].v[k];
              }
            });
            store_bf16x4(p.A + o, a);
            if (p.G) {
              store_bf16x4(p.G + o, v[i]);
              store_bf16x4(p.U + o, w[i]);
            }
            if (p.R)
              *reinterpret_cast<uint32_t*>(p.R + static_cast<size_t>(row) * p.ldr + m) = low_bits4(
                  v[i].v, w[i].v, pack_bf16x2(v[i].v[0], v[i].v[1]), pack_bf16x2(v[i].v[2], v[i].v[3]),
                  pack_bf16x2(w[i].v[0], w[i].v[1]), pack_bf16x2(w[i].v[2], w[i].v[3]));
          } else if constexpr (KIND == kSDown) {
            if (row >= p.T || m >= p.D) continue;
            const size_t o = static_cast<size_t>(row) * p.D + m;
            F4& y = w[i];
            if (p.drop.mode == kDropNone) {
#pragma unroll
              for (int k = 0; k < 4; ++k) y.v[k] += v[i].v[k];
            } else if (p.drop.mode == kDropRandom) {
              auto add = [&](int k, bool kept) {
                if (kept) y.v[k] = fmaf(v[i].v[k], p.drop.scale, y.v[k]);
              };
              const uint64_t e = p.drop.offset + o;
              if (e & 1) for_kept<4, true>(seed, e, p.drop.thr, add);
              else for_kept<4, false>(seed, e, p.drop.thr, add);
            }
            store_bf16x4(p.Y + o, y);
          } else if constexpr (KIND == kSGradAct) {
            if (row >= p.T || m >= p.F) continue;
            const size_t o = static_cast<size_t>(row) * p.ldo + m;
            dispatch_act(p.act, [&](auto act) {
              constexpr int ACT = decltype(act)::value;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float a, d;
                act_eval<ACT, true>(refine(k < 2 ? g_in[i].x : g_in[i].y, halves_g(low[i]), k), a, d);
                const float u = refine(k < 2 ? u_in[i].x : u_in[i].y, halves_u(low[i]), k);
                const float dA = x[i].v[k] * p.scale;
                v[i].v[k] = dA * u * d;
                w[i].v[k] = dA * a;
              }
            });
            store_bf16x4(p.G + o, v[i]);
            store_bf16x4(p.U + o, w[i]);
          } else {
            if (row >= job.rows || m >= job.cols) continue;
            const size_t o = static_cast<size_t>(row) * job.cols + m;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i].v[k] *= job.scale;
            if (job.fp32) {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(job.out) + o);
              if (job.accumulate) {
                const float4 old = *dst;
                v[i].v[0] += old.x, v[i].v[1] += old.y, v[i].v[2] += old.z, v[i].v[3] += old.w;
              }
              *dst = make_float4(v[i].v[0], v[i].v[1], v[i].v[2], v[i].v[3]);
            } else {
              uint16_t* dst = static_cast<uint16_t*>(job.out) + o;
              if (job.accumulate) {
                const F4 old = load_bf16x4(dst);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i].v[k] += old.v[k];
              }
              store_bf16x4(dst, v[i]);
            }
          }
        }
      }
    });
  else if (go && warp == 0 && lane == 0) {
    // timed out: copies in flight get a bounded moment to land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  __syncwarp();
  cluster_sync_all();  // the peers have read this CTA's partial tile
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (p.wait == kWaitLast) pdl_wait();
}

// ------------------------------------------------------------- host side

// launch_pdl with the cluster's size beside it
template <int KIND, int BN>
cudaError_t launch_split_bn(const SplitArgs<KIND>& p, int S, cudaStream_t s) {
  auto kern = k_ffn_split<KIND, BN>;
  const cudaError_t e = prepare_kernel(kern, SplitSmem<BN>::TOTAL);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.job[p.n_jobs - 1].tiles_end) * S);
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = SplitSmem<BN>::TOTAL;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(S), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kern, p, S);
  if (le == cudaSuccess) ++g_kernel_launches;
  return le;
}

template <int KIND>
cudaError_t launch_split(SplitArgs<KIND>& p, const SplitPlan& plan, cudaStream_t s) {
  int end = 0;
  for (int j = 0; j < p.n_jobs; ++j) {
    end += p.job[j].m_tiles * p.job[j].n_tiles;
    p.job[j].tiles_end = end;
  }
  if constexpr (KIND != kSGradW) {  // (dW's N is a feature dimension: always 128)
    if (plan.bn == 16) return launch_split_bn<KIND, 16>(p, plan.cluster, s);
    if (plan.bn == 32) return launch_split_bn<KIND, 32>(p, plan.cluster, s);
    if (plan.bn == 64) return launch_split_bn<KIND, 64>(p, plan.cluster, s);
  }
  return launch_split_bn<KIND, 128>(p, plan.cluster, s);
}

}  // namespace

cudaError_t split_gate_up(const FfnForward& f, const SplitPlan& plan, cudaStream_t s) {
  SplitArgs<kSUp> p = {};
  SplitJob& j = p.job[0];
  const int bn = plan.bn;
  if (!map_kmajor(&j.a[0], f.Wg, f.F, f.D, f.D, 64) || !map_kmajor(&j.a[1], f.Wu, f.F, f.D, f.D, 64) ||
      !map_kmajor(&j.b[0], f.X, f.T, f.D, f.D, bn))
    return cudaErrorInvalidValue;
  j.kb[0] = tiles_of(f.D, BK);
  j.m_tiles = tiles_of(f.F, 64);
  j.n_tiles = tiles_of(f.T, bn);
  p.n_jobs = 1;
  p.wait = kWaitFirst;
  p.T = f.T, p.D = f.D, p.F = f.F, p.act = f.act;
  p.ldo = f.ldo, p.G = f.G, p.U = f.U, p.A = f.A;
  p.R = f.R, p.ldr = f.ldr;
  p.status = f.status;
  return launch_split(p, plan, s);
}

cudaError_t split_down(const FfnForward& f, const SplitPlan& plan, cudaStream_t s) {
  SplitArgs<kSDown> p = {};
  SplitJob& j = p.job[0];
  const int bn = plan.bn;
  if (!map_kmajor(&j.a[0], f.Wd, f.D, f.F, f.F, 128) || !map_kmajor(&j.b[0], f.A, f.T, f.F, f.ldo, bn))
    return cudaErrorInvalidValue;
  j.kb[0] = tiles_of(f.F, BK);
  j.m_tiles = tiles_of(f.D, BM);
  j.n_tiles = tiles_of(f.T, bn);
  p.n_jobs = 1;
  p.wait = kWaitLoadA;  // the gate/up kernel, just before, waited for whatever wrote Wd
  p.T = f.T, p.D = f.D, p.F = f.F;
  p.residual = f.residual, p.Y = f.Y, p.drop = f.drop;
  p.status = f.status;
  return launch_split(p, plan, s);
}

cudaError_t split_grad_act(const FfnBackward& f, const SplitPlan& plan, cudaStream_t s) {
  SplitArgs<kSGradAct> p = {};
  SplitJob& j = p.job[0];
  const int bn = plan.bn;
  if (!map_mnmajor(&j.a[0], f.Wd, f.D, f.F, f.F) || !map_kmajor(&j.b[0], f.dZ, f.T, f.D, f.D, bn))
    return cudaErrorInvalidValue;
  j.kb[0] = tiles_of(f.D, BK);
  j.a_mn = 1;
  j.m_tiles = tiles_of(f.F, BM);
  j.n_tiles = tiles_of(f.T, bn);
  p.n_jobs = 1;
  p.wait = kWaitFirst;
  p.T = f.T, p.D = f.D, p.F = f.F, p.act = f.act, p.scale = f.scale;
  p.G_in = f.G, p.U_in = f.U, p.ldo = f.ldg, p.G = f.dG, p.U = f.dU;
  p.R = const_cast<uint8_t*>(f.R), p.ldr = f.ldr;
  p.status = f.status;
  return launch_split(p, plan, s);
}

cudaError_t split_grad_x(const FfnBackward& f, const SplitPlan& plan, cudaStream_t s) {
  SplitArgs<kSGradX> p = {};
  SplitJob& j = p.job[0];
  const int bn = plan.bn;
  if (!map_mnmajor(&j.a[0], f.Wg, f.F, f.D, f.D) || !map_mnmajor(&j.a[1], f.Wu, f.F, f.D, f.D) ||
      !map_kmajor(&j.b[0], f.dG, f.T, f.F, f.ldg, bn) || !map_kmajor(&j.b[1], f.dU, f.T, f.F, f.ldg, bn))
    return cudaErrorInvalidValue;
  j.kb[0] = j.kb[1] = tiles_of(f.F, BK);
  j.a_mn = 1;
  j.m_tiles = tiles_of(f.D, BM);
  j.n_tiles = tiles_of(f.T, bn);
  j.out = f.dX, j.rows = f.T, j.cols = f.D, j.scale = 1.f;
  p.n_jobs = 1;
  p.wait = kWaitLoadA;  // the kernel just before is this backward's own
  p.status = f.status;
  return launch_split(p, plan, s);
}

// Launched just after split_grad_x or pair_grads' dX, whose output it does not
// touch.
cudaError_t split_grad_w(const FfnBackward& f, const SplitPlan& plan, cudaStream_t s) {
  SplitArgs<kSGradW> p = {};
  const int64_t T = f.T, D = f.D, F = f.F;
  const uint16_t* n_side[3] = {f.dG, f.dU, f.dZ};
  const uint16_t* m_side[3] = {f.X, f.X, f.A};
  const int64_t rows[3] = {F, F, D}, cols[3] = {D, D, F};
  void* out[3] = {f.dWg, f.dWu, f.dWd};
  for (int i = 0; i < 3; ++i) {
    SplitJob& j = p.job[i];
    if (!map_mnmajor(&j.a[0], m_side[i], T, cols[i], cols[i]) ||
        !map_mnmajor(&j.b[0], n_side[i], T, rows[i], i == 2 ? D : f.ldg))
      return cudaErrorInvalidValue;
    j.kb[0] = tiles_of(T, BK);
    j.a_mn = j.b_mn = 1;
    j.m_tiles = tiles_of(cols[i], BM);
    j.n_tiles = tiles_of(rows[i], 128);
    j.out = out[i], j.rows = static_cast<int>(rows[i]), j.cols = static_cast<int>(cols[i]);
    j.scale = i == 2 ? f.scale : 1.f;
    j.fp32 = f.dw_fp32, j.accumulate = f.accumulate;
  }
  p.n_jobs = 3;
  p.wait = kWaitLast;
  p.status = f.status;
  return launch_split(p, plan, s);
}

}  // namespace ss
