// ss_losses.cu -- the losses made of log-probabilities (include/ss_logprob.h):
// clipped policy loss with a KL term, preference pairs, distillation from a
// teacher's top values. Each is one kernel that writes the loss and its gradient.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ss_logprob.cuh"

namespace ss {

namespace {

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool usable(const void* p, uintptr_t a) { return p != nullptr && aligned(p, a); }

constexpr int64_t kMostBlocks = (int64_t(1) << 31) - 1;  // what lies beyond is walked

// N consecutive elements; p null: `none` each
template <int N>
struct Quad {
  float v[N];
};
template <int N>
__device__ __forceinline__ Quad<N> load_quad(const float* p, int64_t i, float none) {
  Quad<N> q;
  if constexpr (N == 4) {
    float4 x = make_float4(none, none, none, none);
    if (p) x = *reinterpret_cast<const float4*>(p + i);
    q.v[0] = x.x, q.v[1] = x.y, q.v[2] = x.z, q.v[3] = x.w;
  } else {
    q.v[0] = p ? p[i] : none;
  }
  return q;
}
template <int N>
__device__ __forceinline__ void store_quad(float* p, int64_t i, const Quad<N>& q) {
  if constexpr (N == 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(q.v[0], q.v[1], q.v[2], q.v[3]);
  else
    p[i] = q.v[0];
}

// ------------------------------------------------------------ policy loss

struct PolicyArgs {
  const float *logp, *old_logp, *advantage, *ref_logp, *weight;
  int64_t n;
  float lo, hi, kl_coef, scale;  // lo, hi: the ends of the clip
  float *loss, *kl, *dlogp;
};

struct PolicyOut {
  float loss, kl, dlogp;
};

// exp(d) - d - 1 from d and e = exp(d) - 1. Near 0, where most tokens of a policy near its
// reference are, e - d is a difference of nearly equal numbers (no digit of it is left at
// |d| = 1e-7); there it is the series d^2 (1/2 + d/6 + d^2/24 + ...), up to d^9 / 9!, whose
// rest is 3e-9 of it at 1/2.
__device__ __forceinline__ float kl_term(float d, float e) {
  if (fabsf(d) < 0.5f) {
    float q = fmaf(d, 1.f / 362880.f, 1.f / 40320.f);
    q = fmaf(d, q, 1.f / 5040.f);
    q = fmaf(d, q, 1.f / 720.f);
    q = fmaf(d, q, 1.f / 120.f);
    q = fmaf(d, q, 1.f / 24.f);
    q = fmaf(d, q, 1.f / 6.f);
    q = fmaf(d, q, 0.5f);
    return d * d * q;
  }
  return e < INFINITY ? e - d : e;  // (not inf - inf)
}

__device__ __forceinline__ PolicyOut policy_token(const PolicyArgs& p, float logp, float old,
                                                  float A, float ref, float m, bool has_ref) {
  PolicyOut o{0.f, 0.f, 0.f};
  if (m == 0.f) return o;
  float gain = 0.f, slope = 0.f;  // of min(r A, clip(r) A)
  if (A != 0.f) {
    const float r = expf(logp - old);
    const float free = r * A, held = fminf(fmaxf(r, p.lo), p.hi) * A;
    gain = held < free ? held : free;
    slope = held < free ? 0.f : free;
  }
  float loss = -gain, d_loss = -slope;
  if (has_ref) {
    const float d = ref - logp, e = expm1f(d);
    o.kl = kl_term(d, e);
    if (p.kl_coef != 0.f) {  // (0 times an infinite term is none)
      loss = fmaf(p.kl_coef, o.kl, loss);
      d_loss = fmaf(-p.kl_coef, e, d_loss);
    }
  }
  o.loss = m * loss;
  o.dlogp = p.scale * (m * d_loss);
  return o;
}

// Memory-bound: 20 bytes read and 12 written a token (with a reference and weights);
// four tokens a thread, 16 bytes an access, where the pointers allow, else one. 2^24
// tokens in 92 us, 5.9 TB/s of the copy's 6.8; two groups a thread, or fewer blocks that
// walk the data, take 93 to 96.
template <bool VEC>
__global__ void __launch_bounds__(256) k_policy_loss(const PolicyArgs p) {
  pdl_enter();
  const bool has_ref = p.ref_logp != nullptr;
  auto tokens = [&](int64_t i, auto count) {
    constexpr int N = decltype(count)::value;
    const Quad<N> x = load_quad<N>(p.logp, i, 0.f), b = load_quad<N>(p.old_logp, i, 0.f),
                  A = load_quad<N>(p.advantage, i, 0.f), r = load_quad<N>(p.ref_logp, i, 0.f),
                  m = load_quad<N>(p.weight, i, 1.f);
    Quad<N> loss, kl, d;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const PolicyOut o = policy_token(p, x.v[j], b.v[j], A.v[j], r.v[j], m.v[j], has_ref);
      loss.v[j] = o.loss, kl.v[j] = o.kl, d.v[j] = o.dlogp;
    }
    store_quad<N>(p.loss, i, loss);
    store_quad<N>(p.dlogp, i, d);
    if (p.kl) store_quad<N>(p.kl, i, kl);
  };
  constexpr int kN = VEC ? 4 : 1;
  const int64_t me = blockIdx.x * int64_t(256) + threadIdx.x, step = int64_t(gridDim.x) * 256;
  for (int64_t g = me; g < p.n / kN; g += step) tokens(g * kN, std::integral_constant<int, kN>{});
  if (VEC && me < (p.n & 3)) tokens((p.n & ~int64_t(3)) + me, std::integral_constant<int, 1>{});
}

// ------------------------------------------------------- preference pairs

struct PreferenceArgs {
  const float *logp, *ref_logp, *weight;
  const int32_t* offsets;
  int pairs, n, kind, average, cluster, vec;
  float beta, smoothing, scale;
  float *loss, *reward, *dlogp;
  int* status;
};

constexpr int kPrefThreads = 256;
constexpr int kPrefMostCluster = 8;

// A number as two floats, hi + lo: 48 bits.
struct Pair {
  float hi, lo;
};

// a + b
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const float s = a.hi + b.hi, v = s - a.hi;
  const float e = (a.hi - (s - v)) + (b.hi - v);  // what s lost
  // (an infinity loses nothing, and the differences above are no numbers then)
  return Pair{s, fabsf(s) < INFINITY ? e + (a.lo + b.lo) : 0.f};
}
template <int LANES>
__device__ __forceinline__ Pair pair_join(Pair v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1)
    v = pair_add(v, Pair{__shfl_xor_sync(0xffffffffu, v.hi, o),
                         __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

// This thread's share of [begin, end), `threads` threads of which it is the me-th, as
// fn(i, step, n, u): u groups of n elements at i, i + step, ...; n is 4 at multiples of
// 4, else 1. Two groups at a time, so that their loads are in flight together.
template <class F>
__device__ __forceinline__ void for_groups(int64_t begin, int64_t end, bool vec, int me,
                                           int threads, F&& fn) {
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, 4> four{};
  const int64_t head = vec ? min((begin + 3) / 4 * 4, end) : end;
  const int64_t tail = vec ? max(end / 4 * 4, head) : end;
  for (int64_t i = begin + me; i < head; i += threads) fn(i, int64_t(0), one, one);
  if (me < end - tail) fn(tail + me, int64_t(0), one, one);
  const int64_t step = 4 * static_cast<int64_t>(threads);
  int64_t i = head + 4 * static_cast<int64_t>(me);
  for (; i + step < tail; i += 2 * step) fn(i, step, four, two);
  for (; i < tail; i += step) fn(i, step, four, one);
}

// a / b for b not 0
__device__ __forceinline__ Pair pair_over(Pair a, Pair b) {
  const float q = a.hi / b.hi;
  const float left = (fmaf(-q, b.hi, a.hi) + a.lo) - q * b.lo;
  return Pair{q, fabsf(q) < INFINITY ? left / b.hi : 0.f};
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  return __uint_as_float(ld_shared_cluster_u32(addr));
}

// A cluster of CTAs per pair: each sums its share of both sequences, the CTAs' sums
// meet in distributed shared memory and are joined in the order of their ranks, each
// CTA makes the loss of them and writes the gradient of its share (the weights are read
// again, from L2). What bounds it is the chain of latencies of the longest pair: 64
// pairs of 2^21 tokens of random lengths take 14.6 us (33 MB, 5 us at the copy rate),
// one of 64 tokens 6.3. A single block of 512 threads per pair took 281 us, clusters of
// 512 threads a CTA, which are not all resident at once, 20.6.
__global__ void __launch_bounds__(kPrefThreads, 6) k_preference_loss(const PreferenceArgs p) {
  static_assert(kPrefThreads >= 128 && 4 * kPrefMostCluster <= 32, "a warp for each sum");
  __shared__ Pair s_warp[kPrefThreads / 32][4];  // sums and weights of both sequences
  __shared__ Pair s_cta[4];
  __shared__ float s_slope[2];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int rank = static_cast<int>(cluster_ctarank()), size = p.cluster;
  const int me = rank * kPrefThreads + static_cast<int>(threadIdx.x);
  const int threads = size * kPrefThreads;
  const int clusters = static_cast<int>(gridDim.x) / size;
  auto in_order = [&](const int (&o)[3]) {
    return o[0] >= 0 && o[1] >= o[0] && o[2] >= o[1] && o[2] <= p.n;
  };
  for (int pair = static_cast<int>(blockIdx.x) / size; pair < p.pairs; pair += clusters) {
    const int o[3] = {p.offsets[2 * pair], p.offsets[2 * pair + 1], p.offsets[2 * pair + 2]};
    if (!in_order(o)) {  // the same for all CTAs
      if (threadIdx.x == 0 && rank == 0) {
        set_status(p.status, SS_ERR_INDEX);
        p.loss[pair] = p.reward[2 * pair] = p.reward[2 * pair + 1] = NAN;
      }
      continue;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      Pair sum{0.f, 0.f}, mass{0.f, 0.f};
      for_groups(o[k], o[k + 1], p.vec, me, threads,
                 [&](int64_t i, int64_t step, auto count, auto groups) {
        constexpr int N = decltype(count)::value, U = decltype(groups)::value;
        Quad<N> m[U], l[U], r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          m[u] = load_quad<N>(p.weight, i + u * step, 1.f);
          l[u] = load_quad<N>(p.logp, i + u * step, 0.f);
          r[u] = load_quad<N>(p.ref_logp, i + u * step, 0.f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float w = m[u].v[j];
            sum = pair_add(sum, Pair{w != 0.f ? w * (l[u].v[j] - r[u].v[j]) : 0.f, 0.f});
            if (p.average) mass = pair_add(mass, Pair{w, 0.f});
          }
      });
      sum = pair_join<32>(sum);
      mass = pair_join<32>(mass);
      if (lane == 0) s_warp[warp][k] = sum, s_warp[warp][2 + k] = mass;
    }
    __syncthreads();
    if (warp < 4) {  // warp k joins the k-th of the four
      constexpr int kWarps = kPrefThreads / 32;
      Pair t = lane < kWarps ? s_warp[lane][warp] : Pair{0.f, 0.f};
      t = pair_join<kWarps>(t);
      if (lane == 0) s_cta[warp] = t;
    }
    __syncthreads();
    if (size > 1) cluster_sync_all();
    if (warp == 0) {
      // lane k + 4 r holds the k-th of rank r; joined over the ranks
      Pair t{0.f, 0.f};
      if (lane < 4 * size) {
        t = s_cta[lane & 3];
        if (size > 1) {
          const uint32_t at = mapa_shared(smem_u32(&s_cta[lane & 3]), lane >> 2);
          t = Pair{ld_cluster_f32(at), ld_cluster_f32(at + 4)};
        }
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        t = pair_add(t, Pair{__shfl_xor_sync(0xffffffffu, t.hi, o),
                             __shfl_xor_sync(0xffffffffu, t.lo, o)});
      const Pair mass{__shfl_sync(0xffffffffu, t.hi, (lane & 1) + 2),
                      __shfl_sync(0xffffffffu, t.lo, (lane & 1) + 2)};
      if (p.average) t = mass.hi != 0.f ? pair_over(t, mass) : Pair{0.f, 0.f};
      const float per = !p.average ? 1.f : mass.hi != 0.f ? 1.f / (mass.hi + mass.lo) : 0.f;
      // lanes 0 and 1: R of the two sequences; the difference in both
      const Pair other{__shfl_xor_sync(0xffffffffu, t.hi, 1), __shfl_xor_sync(0xffffffffu, t.lo, 1)};
      const float sign = (lane & 1) ? -1.f : 1.f;
      const Pair x = pair_add(Pair{sign * t.hi, sign * t.lo}, Pair{-sign * other.hi, -sign * other.lo});
      const float h = p.beta * (x.hi + x.lo);
      float loss, slope;  // slope: d loss / d x
      if (p.kind == SS_PREF_SIGMOID) {
        // log s(h) = min(h, 0) - log(1 + exp(-|h|))
        const float e = expf(-fabsf(h)), l = log1pf(e);
        loss = (1.f - p.smoothing) * (fmaxf(-h, 0.f) + l);
        if (p.smoothing > 0.f) loss += p.smoothing * (fmaxf(h, 0.f) + l);  // (not 0 times inf)
        const float s_neg = h >= 0.f ? e / (1.f + e) : 1.f / (1.f + e);  // s(-h)
        slope = p.beta * (p.smoothing - s_neg);
      } else if (p.kind == SS_PREF_HINGE) {
        loss = fmaxf(0.f, 1.f - h);
        slope = h < 1.f ? -p.beta : 0.f;
        if (isnan(h)) loss = slope = h;
      } else {
        const Pair d = pair_add(x, Pair{-0.5f / p.beta, 0.f});
        const float df = d.hi + d.lo;
        loss = df * df;
        slope = 2.f * df;
      }
      if (lane < 2) {
        s_slope[lane] = sign * p.scale * (slope * per);
        if (rank == 0) p.reward[2 * pair + lane] = p.beta * (t.hi + t.lo);
      }
      if (lane == 0 && rank == 0) p.loss[pair] = loss;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float c = s_slope[k];
      for_groups(o[k], o[k + 1], p.vec, me, threads,
                 [&](int64_t i, int64_t step, auto count, auto groups) {
        constexpr int N = decltype(count)::value, U = decltype(groups)::value;
        Quad<N> m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) m[u] = load_quad<N>(p.weight, i + u * step, 1.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int j = 0; j < N; ++j) m[u].v[j] = m[u].v[j] != 0.f ? m[u].v[j] * c : 0.f;
          store_quad<N>(p.dlogp, i + u * step, m[u]);
        }
      });
    }
    // the peers have read this CTA's sums before the next pair's replace them (or the
    // CTA exits); shared memory is reused by this CTA's own threads too
    if (size > 1) cluster_sync_all();
    else __syncthreads();
  }
  // What lies outside every sequence. The first or last offset of a pair that is bad says
  // nothing of where that is: other pairs' tokens may lie beyond it.
  int64_t begin = p.n, end = p.n;
  if (p.pairs > 0) {
    const int32_t* last = p.offsets + 2 * (static_cast<int64_t>(p.pairs) - 1);
    const int a[3] = {p.offsets[0], p.offsets[1], p.offsets[2]};
    const int b[3] = {last[0], last[1], last[2]};
    begin = in_order(a) ? a[0] : 0;
    end = in_order(b) ? b[2] : p.n;
    if (begin > end) begin = 0, end = p.n;
  }
  const int64_t outside = begin + (p.n - end);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPrefThreads + threadIdx.x; i < outside;
       i += static_cast<int64_t>(gridDim.x) * kPrefThreads)
    p.dlogp[i < begin ? i : i - begin + end] = 0.f;
}

// ---------------------------------------------------------- distillation

struct DistillArgs {
  const float* logp;
  const void* teacher;
  const int32_t* ids;
  const float* weight;
  int T, K, tail;
  float scale;
  float *loss, *dlogp;
};

constexpr float kTailFloor = 1.f / 4096.f;
// a teacher's log-probability up to here is a probability of 0 (the least normal
// number is exp(-87.3))
constexpr float kLeastLog = -87.f;

// What the top ids leave of 1 can be a thousandth, and a rounding of fp32 in their
// sum is then a ten-thousandth of it: with a tail, the exponentials come with their
// roundings and are summed in two parts.

// exp(x) for two x <= 0: x = n log(2) / 2 + r, |r| <= log(2) / 4, with log(2) / 2 in two
// parts (the first has 16 bits, so that n times it is exact) and what the subtraction
// of the second rounds off kept in r_lo; exp(r) = 1 + r + r^2 / 2 + r^3 P(r), what the
// first three terms' sum and the square lose kept too, P the series up to r^7 / 7!,
// whose rest is 2e-11; times the square root of 2, in two parts, where n is odd. Off by
// 3e-10 of the value in all. `top` is a multiple of 2^-23, so that sums of it up to 2
// are exact in fp32; `rest` is what it leaves, below 2^-23.
struct Exp2 {
  float v[2], top[2], rest[2];
};
__device__ __forceinline__ Exp2 exp_pairs(float x0, float x1) {
  const auto both = [](float c) { return f32x2(c, c); };
  const uint64_t x = f32x2(x0 < -87.f ? -87.f : x0, x1 < -87.f ? -87.f : x1);  // (a NaN stays)
  // n by rounding to an integer at 2^23 + 2^22; its low bits then hold it
  constexpr float kMagic = 12582912.f;
  const uint64_t none = both(-1.f);
  const uint64_t m = fma_f32x2(x, both(2.f * 1.4426950408889634f), both(kMagic));
  const uint64_t n = add_f32x2(m, both(-kMagic));
  const uint64_t t = fma_f32x2(n, both(-0x1.62e4p-2f), x);
  const uint64_t r = fma_f32x2(n, both(-0x1.7f7d1cp-21f), t);
  const uint64_t r_lo = fma_f32x2(n, both(-0x1.7f7d1cp-21f), fma_f32x2(r, none, t));
  uint64_t q = fma_f32x2(r, both(1.f / 5040.f), both(1.f / 720.f));
  q = fma_f32x2(q, r, both(1.f / 120.f));
  q = fma_f32x2(q, r, both(1.f / 24.f));
  q = fma_f32x2(q, r, both(1.f / 6.f));
  const uint64_t h = mul_f32x2(r, both(0.5f)), sq = mul_f32x2(h, r);  // r^2 / 2
  const uint64_t sq_lo = fma_f32x2(h, r, mul_f32x2(sq, none));
  const uint64_t one = add_f32x2(r, both(1.f));
  const uint64_t one_lo = fma_f32x2(add_f32x2(one, both(-1.f)), none, r);
  const uint64_t hi = add_f32x2(one, sq);
  const uint64_t hi_lo = fma_f32x2(fma_f32x2(one, none, hi), none, sq);
  uint64_t lo = fma_f32x2(one, r_lo, sq_lo);
  lo = fma_f32x2(mul_f32x2(sq, add_f32x2(r, r)), q, lo);
  lo = add_f32x2(lo, add_f32x2(one_lo, hi_lo));
  float m0, m1;
  f32x2_split(m, m0, m1);
  const int n0 = __float_as_int(m0) - __float_as_int(kMagic);
  const int n1 = __float_as_int(m1) - __float_as_int(kMagic);
  constexpr float kRootHi = 0x1.6a09e6p+0f, kRootLo = 0x1.9fcef4p-26f;
  const uint64_t root = f32x2((n0 & 1) ? kRootHi : 1.f, (n1 & 1) ? kRootHi : 1.f);
  const uint64_t root_lo = f32x2((n0 & 1) ? kRootLo : 0.f, (n1 & 1) ? kRootLo : 0.f);
  const uint64_t p = mul_f32x2(hi, root);
  uint64_t p_lo = fma_f32x2(hi, root, mul_f32x2(p, none));
  p_lo = fma_f32x2(lo, root, fma_f32x2(hi, root_lo, p_lo));
  // 2^floor(n / 2), down to 2^-126
  const uint64_t scale = f32x2(__int_as_float(((n0 >> 1) + 127) << 23),
                               __int_as_float(((n1 >> 1) + 127) << 23));
  float h0, h1, l0, l1;
  f32x2_split(mul_f32x2(p, scale), h0, h1);
  f32x2_split(mul_f32x2(p_lo, scale), l0, l1);
  Exp2 e;
  e.v[0] = h0 + l0, e.v[1] = h1 + l1;
  e.top[0] = (h0 + 1.f) - 1.f, e.top[1] = (h1 + 1.f) - 1.f;
  e.rest[0] = (h0 - e.top[0]) + l0, e.rest[1] = (h1 - e.top[1]) + l1;
  return e;
}

// Four entries of a token, those that are not there absent.
template <bool BF16, bool VEC>
struct Entries {
  float l[4], x[4], m;
  unsigned on;  // bit i: entry i is there
  __device__ __forceinline__ void load(const DistillArgs& p, int64_t t, int k0) {
    const bool valid = t < p.T;
    const int64_t at = t * p.K + k0;
    const int nk = valid ? min(max(p.K - k0, 0), 4) : 0;
    m = valid ? (p.weight ? p.weight[t] : 1.f) : 0.f;
    on = 0u;
    if (VEC && nk == 4) {
      const float4 a = *reinterpret_cast<const float4*>(p.logp + at);
      l[0] = a.x, l[1] = a.y, l[2] = a.z, l[3] = a.w;
      if (BF16) {
        const uint2 b =
            *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.teacher) + at);
        x[0] = __uint_as_float(b.x << 16), x[1] = __uint_as_float(b.x & 0xffff0000u);
        x[2] = __uint_as_float(b.y << 16), x[3] = __uint_as_float(b.y & 0xffff0000u);
      } else {
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p.teacher) + at);
        x[0] = b.x, x[1] = b.y, x[2] = b.z, x[3] = b.w;
      }
      on = 15u;
      if (p.ids) {
        const int4 id = *reinterpret_cast<const int4*>(p.ids + at);
        on = (id.x >= 0 ? 1u : 0u) | (id.y >= 0 ? 2u : 0u) | (id.z >= 0 ? 4u : 0u) |
             (id.w >= 0 ? 8u : 0u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        l[i] = x[i] = 0.f;
        if (i >= nk) continue;
        on |= !p.ids || p.ids[at + i] >= 0 ? 1u << i : 0u;
        l[i] = p.logp[at + i];
        x[i] = BF16 ? __uint_as_float(
                          static_cast<uint32_t>(static_cast<const uint16_t*>(p.teacher)[at + i])
                          << 16)
                    : static_cast<const float*>(p.teacher)[at + i];
      }
    }
  }
};

// A token's K entries over LANES lanes, four a lane. The instructions bound it, not the
// 14 bytes an entry: 65536 tokens of K 128 in 26 us, 40 with a tail (3.4 of 4 possible
// instructions a cycle, most of them the exponentials'), where a copy of as many bytes
// takes 17. Two or four times as many entries a lane, which halve the steps of each
// sum over lanes, take registers that cost more (36 and 39 us without a tail); the
// next token's entries loaded ahead took 45 us with a tail.
template <int LANES, bool BF16, bool VEC>
__global__ void __launch_bounds__(256, 5) k_distill_loss(const DistillArgs p) {
  pdl_enter();
  const int64_t lanes = (static_cast<int64_t>(p.T) * LANES + 255) / 256 * 256;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int k0 = static_cast<int>(first % LANES) * 4;
  // the same trip count for every lane of a block
  for (int64_t g = first; g < lanes; g += step) {
    const int64_t t = g / LANES;
    Entries<BF16, VEC> now;
    now.load(p, t, k0);
    float (&l)[4] = now.l, (&x)[4] = now.x;
    const float m = now.m;
    const bool here[4] = {(now.on & 1u) != 0u, (now.on & 2u) != 0u, (now.on & 4u) != 0u,
                          (now.on & 8u) != 0u};
    auto join = [](float v) {
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
    float extra = 0.f, loss = 0.f;
    const unsigned mine = (0xffffffffu >> (32 - LANES)) << (threadIdx.x & 31 & ~(LANES - 1));
    const bool used = (__ballot_sync(0xffffffffu, now.on != 0u) & mine) != 0u && m != 0.f;
    // l becomes the slope
    if (p.tail) {
      float sp[2] = {0.f, 0.f}, sq[2] = {0.f, 0.f}, q[4];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const Exp2 a = exp_pairs(x[i], x[i + 1]), b = exp_pairs(l[i], l[i + 1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool on = here[i + j], known = on && !(x[i + j] <= kLeastLog);
          const float pr = known ? a.v[j] : 0.f;
          q[i + j] = on ? b.v[j] : 0.f;
          sp[0] += known ? a.top[j] : 0.f, sp[1] += known ? a.rest[j] : 0.f;
          sq[0] += on ? b.top[j] : 0.f, sq[1] += on ? b.rest[j] : 0.f;
          if (known) loss += pr * (x[i + j] - l[i + j]);
          x[i + j] = pr;
        }
      }
      loss = join(loss);
      const float left = (1.f - join(sp[0])) - join(sp[1]), p1 = left < 0.f ? 0.f : left;
      const float rest = (1.f - join(sq[0])) - join(sq[1]);
      const float q1 = rest < kTailFloor ? kTailFloor : rest;  // (a NaN stays in both)
      if (p1 != 0.f) extra = p1 * (logf(p1) - logf(q1));
      const float ratio = rest <= kTailFloor ? 0.f : p1 / q1;
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] = fmaf(ratio, q[i], -x[i]);
    } else {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = here[i] ? fmaxf(top, x[i]) : top;
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // sum of exp(x - top); and, with log p = x - top - log(sum), of exp(x - top)
      // times (x - top - l), from which the loss is made. Where no value is a number above
      // -infinity, top is -infinity: -infinity counts as 0 there too, a NaN stays one
      float sum = 0.f, part = 0.f, pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float d = x[i] - top;
        pr[i] = here[i] && x[i] != -INFINITY ? expf(d) : 0.f;
        sum += pr[i];
        if (pr[i] > 0.f) part += pr[i] * (d - l[i]);
      }
      sum = join(sum);
      part = join(part);
      const float per = sum != 0.f ? 1.f / sum : 0.f;  // (a NaN stays)
      loss = part * per;
      if (sum > 0.f) extra = -logf(sum);
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] = -per * pr[i];
    }
    loss += extra;
    if (t >= p.T) continue;
    const int64_t at = t * p.K + k0;
    const int nk = min(max(p.K - k0, 0), 4);
    if (k0 == 0) p.loss[t] = used ? m * loss : 0.f;
    const float scale = p.scale * m;
    float d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = used && here[i] ? scale * l[i] : 0.f;
    if (VEC && nk == 4) {
      *reinterpret_cast<float4*>(p.dlogp + at) = make_float4(d[0], d[1], d[2], d[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < nk) p.dlogp[at + i] = d[i];
    }
  }
}

template <int LANES>
cudaError_t distill(const DistillArgs& p, bool bf16, bool vec, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(p.T) * LANES + 255) / 256;
  const dim3 grid(static_cast<unsigned>(std::min(blocks, kMostBlocks)));
  if (bf16)
    return vec ? launch_pdl(k_distill_loss<LANES, true, true>, grid, dim3(256), 0, s, p)
               : launch_pdl(k_distill_loss<LANES, true, false>, grid, dim3(256), 0, s, p);
  return vec ? launch_pdl(k_distill_loss<LANES, false, true>, grid, dim3(256), 0, s, p)
             : launch_pdl(k_distill_loss<LANES, false, false>, grid, dim3(256), 0, s, p);
}

}  // namespace

}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_policy_loss(const float* logp, const float* old_logp, const float* advantage,
                         const float* ref_logp, const float* weight, int64_t n, float clip_low,
                         float clip_high, float kl_coef, float scale, float* loss, float* kl,
                         float* dlogp, ss_stream stream) {
  if (n < 0 || !(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) ||
      !(kl_coef >= 0.f) || !std::isfinite(kl_coef) || !std::isfinite(scale) ||
      (!ref_logp && (kl_coef != 0.f || kl)))
    return SS_ERR_INVALID;
  if (n >= (int64_t(1) << 62)) return SS_ERR_UNSUPPORTED;
  if (n == 0) return SS_OK;
  if (!usable(logp, 4) || !usable(old_logp, 4) || !usable(advantage, 4) || !aligned(ref_logp, 4) ||
      !aligned(weight, 4) || !usable(loss, 4) || !aligned(kl, 4) || !usable(dlogp, 4))
    return SS_ERR_INVALID;
  const int nsm = current_num_sms();
  if (nsm <= 0) return record_failure("cudaGetDevice/cudaDeviceGetAttribute", cudaGetLastError());
  const PolicyArgs p{logp, old_logp, advantage, ref_logp, weight, n, 1.f - clip_low,
                     1.f + clip_high, kl_coef, scale, loss, kl, dlogp};
  const bool vec = aligned(logp, 16) && aligned(old_logp, 16) && aligned(advantage, 16) &&
                   aligned(ref_logp, 16) && aligned(weight, 16) && aligned(loss, 16) &&
                   aligned(kl, 16) && aligned(dlogp, 16);
  const int64_t each = vec ? 256 * 4 : 256;
  const dim3 grid(static_cast<unsigned>(std::min((n + each - 1) / each, kMostBlocks)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  StageTrace trace(s, "policy_loss");
  const cudaError_t e = vec ? launch_pdl(k_policy_loss<true>, grid, dim3(256), 0, s, p)
                            : launch_pdl(k_policy_loss<false>, grid, dim3(256), 0, s, p);
  return e == cudaSuccess ? SS_OK : record_failure("launch k_policy_loss", e);
}

ss_status ss_preference_loss(const float* logp, const float* ref_logp, const float* weight,
                             const int32_t* offsets, int64_t pairs, int64_t n, int kind,
                             float beta, float smoothing, int average, float scale, float* loss,
                             float* reward, float* dlogp, void* workspace,
                             size_t workspace_bytes, ss_stream stream) {
  if (n < 0 || pairs < 0 || kind < SS_PREF_SIGMOID || kind > SS_PREF_IPO || !(beta > 0.f) ||
      !std::isfinite(beta) || !(smoothing >= 0.f && smoothing <= 0.5f) ||
      (smoothing != 0.f && kind != SS_PREF_SIGMOID) || (average != 0 && average != 1) ||
      !std::isfinite(scale))
    return SS_ERR_INVALID;
  if (n >= (int64_t(1) << 31) || pairs >= (int64_t(1) << 29)) return SS_ERR_UNSUPPORTED;
  if (pairs == 0 && n == 0) return SS_OK;
  if (!usable(workspace, 16) || (n > 0 && (!usable(logp, 4) || !usable(dlogp, 4))) ||
      !aligned(ref_logp, 4) || !aligned(weight, 4) ||
      (pairs > 0 && (!usable(offsets, 4) || !usable(loss, 4) || !usable(reward, 4))))
    return SS_ERR_INVALID;
  if (workspace_bytes < kHeaderBytes) return SS_ERR_WORKSPACE;
  const int nsm = current_num_sms();
  if (nsm <= 0) return record_failure("cudaGetDevice/cudaDeviceGetAttribute", cudaGetLastError());
  PreferenceArgs p{};
  p.logp = logp, p.ref_logp = ref_logp, p.weight = weight, p.offsets = offsets;
  p.pairs = static_cast<int>(pairs), p.n = static_cast<int>(n);
  p.kind = kind, p.average = average;
  p.beta = beta, p.smoothing = smoothing, p.scale = scale;
  p.loss = loss, p.reward = reward, p.dlogp = dlogp;
  p.status = static_cast<int*>(workspace);
  p.vec = aligned(logp, 16) && aligned(ref_logp, 16) && aligned(weight, 16) && aligned(dlogp, 16);
  // a CTA per 4096 tokens of a pair of average length, up to the largest portable
  // cluster; pairs beyond the resident clusters take turns
  const int64_t each = n / std::max<int64_t>(pairs, 1);
  p.cluster = 1;
  while (p.cluster < kPrefMostCluster && each > 4096 * int64_t(p.cluster)) p.cluster *= 2;
  const int64_t ctas = std::min<int64_t>(std::max<int64_t>(pairs, 1) * p.cluster, int64_t(nsm) * 4);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  StageTrace trace(s, "preference_loss");
  cudaError_t e = prepare_kernel(k_preference_loss, 0);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas / p.cluster * p.cluster));
    cfg.blockDim = dim3(kPrefThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(p.cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, k_preference_loss, p);
    if (e == cudaSuccess) ++g_kernel_launches;
  }
  return e == cudaSuccess ? SS_OK : record_failure("launch k_preference_loss", e);
}

ss_status ss_distill_loss(const float* logp, const void* teacher, int teacher_dtype,
                          const int32_t* ids, const float* weight, int64_t T, int64_t K, int tail,
                          float scale, float* loss, float* dlogp, ss_stream stream) {
  if (T < 0 || K < 1 || (teacher_dtype != SS_BF16 && teacher_dtype != SS_FP32) ||
      (tail != 0 && tail != 1) || !std::isfinite(scale))
    return SS_ERR_INVALID;
  if (T >= (int64_t(1) << 31) || K > SS_MAX_IDS) return SS_ERR_UNSUPPORTED;
  if (T == 0) return SS_OK;
  const bool bf16 = teacher_dtype == SS_BF16;
  if (!usable(logp, 4) || !usable(teacher, bf16 ? 2 : 4) || !aligned(ids, 4) ||
      !aligned(weight, 4) || !usable(loss, 4) || !usable(dlogp, 4))
    return SS_ERR_INVALID;
  const int nsm = current_num_sms();
  if (nsm <= 0) return record_failure("cudaGetDevice/cudaDeviceGetAttribute", cudaGetLastError());
  const DistillArgs p{logp, teacher, ids, weight, static_cast<int>(T), static_cast<int>(K), tail,
                      scale, loss, dlogp};
  const bool vec = K % 4 == 0 && aligned(logp, 16) && aligned(teacher, bf16 ? 8 : 16) &&
                   aligned(ids, 16) && aligned(dlogp, 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  StageTrace trace(s, "distill_loss");
  const cudaError_t e = K <= 4    ? distill<1>(p, bf16, vec, s)
                        : K <= 8  ? distill<2>(p, bf16, vec, s)
                        : K <= 16 ? distill<4>(p, bf16, vec, s)
                        : K <= 32 ? distill<8>(p, bf16, vec, s)
                        : K <= 64 ? distill<16>(p, bf16, vec, s)
                                  : distill<32>(p, bf16, vec, s);
  return e == cudaSuccess ? SS_OK : record_failure("launch k_distill_loss", e);
}

}  // extern "C"
