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
    o.kl = e - d;
    loss = fmaf(p.kl_coef, o.kl, loss);
    d_loss = fmaf(-p.kl_coef, e, d_loss);
  }
  o.loss = m * loss;
  o.dlogp = p.scale * (m * d_loss);
  return o;
}

// Memory-bound: 20 bytes read and 12 written a token (with a reference and
// weights). VEC tokens a thread, 16 bytes an access where the pointers allow.
template <int VEC>
__global__ void __launch_bounds__(256) k_policy_loss(const PolicyArgs p) {
  pdl_enter();
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  const bool has_ref = p.ref_logp != nullptr;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; g * VEC < p.n; g += step) {
    const int64_t i = g * VEC;
    if (VEC == 4 && i + 4 <= p.n) {
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f), u = make_float4(1.f, 1.f, 1.f, 1.f);
      const float4 x = *reinterpret_cast<const float4*>(p.logp + i);
      const float4 b = *reinterpret_cast<const float4*>(p.old_logp + i);
      const float4 A = *reinterpret_cast<const float4*>(p.advantage + i);
      const float4 r = has_ref ? *reinterpret_cast<const float4*>(p.ref_logp + i) : z;
      const float4 m = p.weight ? *reinterpret_cast<const float4*>(p.weight + i) : u;
      const PolicyOut o0 = policy_token(p, x.x, b.x, A.x, r.x, m.x, has_ref);
      const PolicyOut o1 = policy_token(p, x.y, b.y, A.y, r.y, m.y, has_ref);
      const PolicyOut o2 = policy_token(p, x.z, b.z, A.z, r.z, m.z, has_ref);
      const PolicyOut o3 = policy_token(p, x.w, b.w, A.w, r.w, m.w, has_ref);
      *reinterpret_cast<float4*>(p.loss + i) = make_float4(o0.loss, o1.loss, o2.loss, o3.loss);
      *reinterpret_cast<float4*>(p.dlogp + i) = make_float4(o0.dlogp, o1.dlogp, o2.dlogp, o3.dlogp);
      if (p.kl) *reinterpret_cast<float4*>(p.kl + i) = make_float4(o0.kl, o1.kl, o2.kl, o3.kl);
    } else {
      for (int64_t j = i; j < std::min<int64_t>(i + VEC, p.n); ++j) {
        const PolicyOut o =
            policy_token(p, p.logp[j], p.old_logp[j], p.advantage[j],
                         has_ref ? p.ref_logp[j] : 0.f, p.weight ? p.weight[j] : 1.f, has_ref);
        p.loss[j] = o.loss;
        p.dlogp[j] = o.dlogp;
        if (p.kl) p.kl[j] = o.kl;
      }
    }
  }
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

constexpr int kPrefThreads = 512;

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

// fn(i, n) for the elements i .. i + n - 1 (n = 4 at a multiple of 4, else 1) of this
// thread's share of [begin, end): `threads` threads, of which it is the me-th.
template <class F>
__device__ __forceinline__ void for_quads(int64_t begin, int64_t end, bool vec, int me,
                                          int threads, F&& fn) {
  if (!vec) {
    for (int64_t i = begin + me; i < end; i += threads) fn(i, std::integral_constant<int, 1>{});
    return;
  }
  const int64_t head = min((begin + 3) / 4 * 4, end), tail = max(end / 4 * 4, head);
  if (me < head - begin) fn(begin + me, std::integral_constant<int, 1>{});
  if (me < end - tail) fn(tail + me, std::integral_constant<int, 1>{});
  for (int64_t i = head + 4 * static_cast<int64_t>(me); i < tail;
       i += 4 * static_cast<int64_t>(threads))
    fn(i, std::integral_constant<int, 4>{});
}

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

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  return __uint_as_float(ld_shared_cluster_u32(addr));
}

// A cluster of CTAs per pair: each sums its share of both sequences, the CTAs' sums
// meet in distributed shared memory in the order of their ranks, each CTA makes the
// loss of them and writes the gradient of its share (the weights are read again, from
// L2). 64 pairs of 32768 tokens on average, with reference and weights: a block alone
// per pair took 281 us.
__global__ void __launch_bounds__(kPrefThreads) k_preference_loss(const PreferenceArgs p) {
  __shared__ Pair s_warp[kPrefThreads / 32][4];  // sums and weights of both sequences
  __shared__ Pair s_cta[4];
  __shared__ float s_slope[2];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int rank = static_cast<int>(cluster_ctarank()), size = p.cluster;
  const int me = rank * kPrefThreads + static_cast<int>(threadIdx.x);
  const int threads = size * kPrefThreads;
  const int clusters = static_cast<int>(gridDim.x) / size;
  for (int pair = static_cast<int>(blockIdx.x) / size; pair < p.pairs; pair += clusters) {
    const int o[3] = {p.offsets[2 * pair], p.offsets[2 * pair + 1], p.offsets[2 * pair + 2]};
    if (o[0] < 0 || o[1] < o[0] || o[2] < o[1] || o[2] > p.n) {  // the same for all CTAs
      if (threadIdx.x == 0 && rank == 0) {
        set_status(p.status, SS_ERR_INDEX);
        p.loss[pair] = p.reward[2 * pair] = p.reward[2 * pair + 1] = NAN;
      }
      continue;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      Pair sum{0.f, 0.f}, mass{0.f, 0.f};
      for_quads(o[k], o[k + 1], p.vec, me, threads, [&](int64_t i, auto count) {
        constexpr int N = decltype(count)::value;
        const Quad<N> m = load_quad<N>(p.weight, i, 1.f), l = load_quad<N>(p.logp, i, 0.f),
                      r = load_quad<N>(p.ref_logp, i, 0.f);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float x = m.v[j] != 0.f ? m.v[j] * (l.v[j] - r.v[j]) : 0.f;
          sum = pair_add(sum, Pair{x, 0.f});
          mass = pair_add(mass, Pair{m.v[j], 0.f});
        }
      });
      sum = pair_join<32>(sum);
      mass = pair_join<32>(mass);
      if (lane == 0) s_warp[warp][k] = sum, s_warp[warp][2 + k] = mass;
    }
    __syncthreads();
    if (threadIdx.x < 4) {
      Pair t = s_warp[0][threadIdx.x];
      for (int w = 1; w < kPrefThreads / 32; ++w) t = pair_add(t, s_warp[w][threadIdx.x]);
      s_cta[threadIdx.x] = t;
    }
    __syncthreads();
    if (size > 1) cluster_sync_all();
    if (threadIdx.x == 0) {
      double t[4];
      for (int k = 0; k < 4; ++k) {
        Pair all{0.f, 0.f};
        for (int r = 0; r < size; ++r) {
          Pair v = s_cta[k];
          if (size > 1) {
            const uint32_t at = mapa_shared(smem_u32(&s_cta[k]), r);
            v = Pair{ld_cluster_f32(at), ld_cluster_f32(at + 4)};
          }
          all = pair_add(all, v);
        }
        t[k] = static_cast<double>(all.hi) + static_cast<double>(all.lo);
      }
      double per[2] = {1., 1.};
      if (p.average)
        for (int k = 0; k < 2; ++k) per[k] = t[2 + k] != 0. ? 1. / t[2 + k] : 0.;
      const double r0 = t[0] * per[0], r1 = t[1] * per[1], x = r0 - r1;
      const double h = p.beta * x;
      float loss, slope;  // slope: d loss / d x
      if (p.kind == SS_PREF_SIGMOID) {
        // log s(h) = min(h, 0) - log(1 + exp(-|h|))
        const float hf = static_cast<float>(h), e = expf(-fabsf(hf)), l = log1pf(e);
        loss = (1.f - p.smoothing) * (fmaxf(-hf, 0.f) + l) + p.smoothing * (fmaxf(hf, 0.f) + l);
        const float s_neg = hf >= 0.f ? e / (1.f + e) : 1.f / (1.f + e);  // s(-h)
        slope = p.beta * (p.smoothing - s_neg);
      } else if (p.kind == SS_PREF_HINGE) {
        loss = static_cast<float>(fmax(0., 1. - h));
        slope = h < 1. ? -p.beta : 0.f;
      } else {
        const double d = x - 0.5 / p.beta;
        loss = static_cast<float>(d * d);
        slope = static_cast<float>(2. * d);
      }
      if (rank == 0) {
        p.loss[pair] = loss;
        p.reward[2 * pair] = static_cast<float>(p.beta * r0);
        p.reward[2 * pair + 1] = static_cast<float>(p.beta * r1);
      }
      s_slope[0] = static_cast<float>(p.scale * (slope * per[0]));
      s_slope[1] = static_cast<float>(-p.scale * (slope * per[1]));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float c = s_slope[k];
      for_quads(o[k], o[k + 1], p.vec, me, threads, [&](int64_t i, auto count) {
        constexpr int N = decltype(count)::value;
        Quad<N> m = load_quad<N>(p.weight, i, 1.f);
#pragma unroll
        for (int j = 0; j < N; ++j) m.v[j] = m.v[j] != 0.f ? m.v[j] * c : 0.f;
        store_quad<N>(p.dlogp, i, m);
      });
    }
    // the peers have read this CTA's sums before the next pair's replace them (or the
    // CTA exits); shared memory is reused by this CTA's own threads too
    if (size > 1) cluster_sync_all();
    else __syncthreads();
  }
  // what lies outside every sequence
  const int64_t begin = p.pairs > 0 ? min(max(p.offsets[0], 0), p.n) : p.n;
  const int64_t end = p.pairs > 0 ? min(max(p.offsets[2 * p.pairs], static_cast<int>(begin)), p.n)
                                  : p.n;
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

// What the top ids leave of 1 can be a thousandth, and a rounding of fp32 in their
// sum is then a ten-thousandth of it: with a tail, the exponentials and their sums
// are pairs of floats.

// exp(x) for x <= 0: x = n log 2 + r, |r| <= log(2) / 2, with log 2 in two parts (the
// first has 16 bits, so that n times it is exact) and what the subtraction of the
// second rounds off kept in r_lo; exp(r) = 1 + r + r^2 / 2 + r^3 P(r), what the
// first three terms' sum and the square lose kept too, P the series up to r^8 / 8!,
// whose rest is 2e-10.
__device__ __forceinline__ Pair exp_pair(float x) {
  constexpr float c1 = 0x1.62e4p-1f, c2 = 0x1.7f7d1cp-20f;
  x = fmaxf(x, -100.f);
  const float n = rintf(x * 1.4426950408889634f);
  const float t = fmaf(-n, c1, x);
  const float r = fmaf(-n, c2, t), r_lo = fmaf(-n, c2, t - r);
  float q = 1.f / 40320.f;
  q = fmaf(q, r, 1.f / 5040.f);
  q = fmaf(q, r, 1.f / 720.f);
  q = fmaf(q, r, 1.f / 120.f);
  q = fmaf(q, r, 1.f / 24.f);
  q = fmaf(q, r, 1.f / 6.f);
  const float h = 0.5f * r, sq = h * r, sq_lo = fmaf(h, r, -sq);  // r^2 / 2
  const float one = 1.f + r, one_lo = r - (one - 1.f);
  const float hi = one + sq, hi_lo = sq - (hi - one);
  const float lo = (one_lo + hi_lo) + fmaf(sq * (2.f * r), q, fmaf(one, r_lo, sq_lo));
  // 2^n, 0 below the normal numbers
  const float scale = n >= -126.f ? __int_as_float((127 + static_cast<int>(n)) << 23) : 0.f;
  return Pair{hi * scale, lo * scale};
}

// A token's K entries over LANES lanes, four each.
template <int LANES, bool BF16, bool VEC>
__global__ void __launch_bounds__(256) k_distill_loss(const DistillArgs p) {
  pdl_enter();
  const int64_t lanes = static_cast<int64_t>(p.T) * LANES;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  // the same trip count for every lane of a warp
  for (int64_t g0 = static_cast<int64_t>(blockIdx.x) * 256; g0 < lanes; g0 += step) {
    const int64_t g = g0 + threadIdx.x;
    const bool valid = g < lanes;
    const int64_t t = valid ? g / LANES : 0;
    const int k0 = static_cast<int>(g % LANES) * 4;
    const int64_t at = t * p.K + k0;
    const int nk = valid ? min(max(p.K - k0, 0), 4) : 0;
    float l[4], x[4];
    bool here[4];
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
      int4 id = make_int4(0, 0, 0, 0);
      if (p.ids) id = *reinterpret_cast<const int4*>(p.ids + at);
      here[0] = id.x >= 0, here[1] = id.y >= 0, here[2] = id.z >= 0, here[3] = id.w >= 0;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        here[i] = i < nk && (!p.ids || p.ids[at + i] >= 0);
        l[i] = i < nk ? p.logp[at + i] : 0.f;
        x[i] = 0.f;
        if (i < nk)
          x[i] = BF16 ? __uint_as_float(
                            static_cast<uint32_t>(static_cast<const uint16_t*>(p.teacher)[at + i])
                            << 16)
                      : static_cast<const float*>(p.teacher)[at + i];
      }
    }
    const float m = valid ? (p.weight ? p.weight[t] : 1.f) : 0.f;
    auto join = [](float v) {
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
    auto rest_of_1 = [](Pair v) {
      v = pair_join<LANES>(v);
      return (1.f - v.hi) - v.lo;
    };
    float pr[4], extra = 0.f, ratio = 0.f, loss = 0.f;
    float any = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) any = here[i] ? 1.f : any;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) any = fmaxf(any, __shfl_xor_sync(0xffffffffu, any, o));
    const bool used = m != 0.f && any != 0.f;
    if (p.tail) {
      Pair sp{0.f, 0.f}, sq{0.f, 0.f};
      float q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair a = here[i] ? exp_pair(x[i]) : Pair{0.f, 0.f};
        const Pair b = here[i] ? exp_pair(l[i]) : Pair{0.f, 0.f};
        pr[i] = a.hi + a.lo;
        q[i] = b.hi + b.lo;
        sp = pair_add(sp, a);
        sq = pair_add(sq, b);
        if (pr[i] > 0.f) loss += pr[i] * (x[i] - l[i]);
      }
      const float p1 = fmaxf(rest_of_1(sp), 0.f);
      const float rest = rest_of_1(sq), q1 = fmaxf(rest, kTailFloor);
      if (p1 > 0.f) extra = p1 * (logf(p1) - logf(q1));
      ratio = rest > kTailFloor ? p1 / q1 : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] = fmaf(ratio, q[i], -pr[i]);  // the slope
    } else {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = here[i] ? fmaxf(top, x[i]) : top;
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      float sp = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pr[i] = here[i] && top > -INFINITY ? expf(x[i] - top) : 0.f;
        sp += pr[i];
      }
      sp = join(sp);
      const float per = sp > 0.f ? 1.f / sp : 0.f, ls = top + logf(sp);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pr[i] *= per;
        if (pr[i] > 0.f) loss += pr[i] * ((x[i] - ls) - l[i]);
        l[i] = -pr[i];
      }
    }
    loss = join(loss) + extra;
    if (!valid) continue;
    if (k0 == 0) p.loss[t] = used ? m * loss : 0.f;
    const float c = p.scale * m;
    float d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = used && here[i] ? c * l[i] : 0.f;
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
cudaError_t distill(const DistillArgs& p, bool bf16, bool vec, int num_sms, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(p.T) * LANES + 255) / 256;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(blocks, int64_t(num_sms) * 32)));
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
  const int64_t items = vec ? (n + 3) / 4 : n;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((items + 255) / 256, int64_t(nsm) * 32)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  StageTrace trace(s, "policy_loss");
  const cudaError_t e = vec ? launch_pdl(k_policy_loss<4>, grid, dim3(256), 0, s, p)
                            : launch_pdl(k_policy_loss<1>, grid, dim3(256), 0, s, p);
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
  while (p.cluster < 8 && each > 4096 * int64_t(p.cluster)) p.cluster = std::max(1, 2 * p.cluster);
  p.cluster = std::max(1, p.cluster);
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
  const cudaError_t e = K <= 4    ? distill<1>(p, bf16, vec, nsm, s)
                        : K <= 8  ? distill<2>(p, bf16, vec, nsm, s)
                        : K <= 16 ? distill<4>(p, bf16, vec, nsm, s)
                        : K <= 32 ? distill<8>(p, bf16, vec, nsm, s)
                        : K <= 64 ? distill<16>(p, bf16, vec, nsm, s)
                                  : distill<32>(p, bf16, vec, nsm, s);
  return e == cudaSuccess ? SS_OK : record_failure("launch k_distill_loss", e);
}

}  // extern "C"
