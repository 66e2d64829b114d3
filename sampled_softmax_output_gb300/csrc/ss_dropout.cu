// ss_dropout.cu -- dropout and its gradient as one pass over the data:
//   y = residual + (kept ? scale * x : 0)
// The mask comes from ss_dropout.cuh and is stored nowhere.
//
// Bound by memory: 4 bytes an element in bf16 (6 with a residual). Next to
// that stand about 11 integer instructions an element for the hash. Groups of
// 8 elements keep every access 16 bytes wide, and two groups per thread are in
// flight before the first is hashed.
#include "ss_ffn.cuh"

namespace ss {

namespace {

constexpr int kDropThreads = 256;
constexpr int kDropGroups = 2;  // groups of 8 elements in flight per thread

struct Vec8 {
  float v[8];
};

__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  Vec8 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    r.v[2 * k] = __uint_as_float(w[k] << 16);
    r.v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ Vec8 load8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(uint16_t* p, const Vec8& r) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]),
                 pack_bf16x2(r.v[4], r.v[5]), pack_bf16x2(r.v[6], r.v[7]));
}
__device__ __forceinline__ void store8(float* p, const Vec8& r) {
  reinterpret_cast<float4*>(p)[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
}
__device__ __forceinline__ float load1(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = bf16_bits(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// residual + what dropout leaves of x (without a residual, a dropped element
// is +0 and a kept one keeps its sign of zero)
template <bool RES>
__device__ __forceinline__ float drop_one(float x, float r, bool kept, float scale) {
  if (RES) return kept ? fmaf(x, scale, r) : r;
  return kept ? x * scale : 0.f;
}

// One element, by itself: unaligned buffers and the tail of a length that is
// not a multiple of 8.
template <class T, bool RES>
__device__ __forceinline__ void drop_element(const T* x, const T* res, T* y, int64_t i,
                                             const DropArgs& d, uint64_t seed) {
  const uint64_t e = d.offset + static_cast<uint64_t>(i);
  bool kept = d.mode == kDropNone;
  if (d.mode == kDropRandom) {
    const uint64_t h = splitmix_out(seed + ((e >> 1) + 1) * kSplitMixGamma);
    kept = static_cast<uint32_t>((e & 1) ? h >> 32 : h) >= d.thr;
  }
  store1(y + i, drop_one<RES>(load1(x + i), RES ? load1(res + i) : 0.f, kept, d.scale));
}

// 16-byte aligned buffers; y may be x or residual (each element is read by the
// thread that writes it, before it writes).
template <class T, bool RES, bool ODD>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout(const T* x, const T* res, int64_t n, const DropArgs d, T* y) {
  pdl_enter();
  const uint64_t seed = drop_seed(d);
  const int64_t n8 = n >> 3;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kDropThreads;
  int64_t g = static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x;
  if (g < (n & 7)) drop_element<T, RES>(x, res, y, (n8 << 3) + g, d, seed);
  for (; g < n8; g += kDropGroups * step) {
    Vec8 a[kDropGroups], r[kDropGroups];
#pragma unroll
    for (int u = 0; u < kDropGroups; ++u) {
      const int64_t at = (g + u * step) << 3;
      if (g + u * step < n8) {
        a[u] = load8(x + at);
        if (RES) r[u] = load8(res + at);
      }
    }
#pragma unroll
    for (int u = 0; u < kDropGroups; ++u) {
      if (g + u * step >= n8) break;
      const int64_t at = (g + u * step) << 3;
      if (d.mode == kDropRandom) {
        for_kept<8, ODD>(seed, d.offset + static_cast<uint64_t>(at), d.thr, [&](int i, bool kept) {
          a[u].v[i] = drop_one<RES>(a[u].v[i], r[u].v[i], kept, d.scale);
        });
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          a[u].v[i] = drop_one<RES>(a[u].v[i], r[u].v[i], d.mode == kDropNone, d.scale);
      }
      store8(y + at, a[u]);
    }
  }
}

template <class T, bool RES>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout_unaligned(const T* x, const T* res, int64_t n, const DropArgs d, T* y) {
  pdl_enter();
  const uint64_t seed = drop_seed(d);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kDropThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x; i < n; i += step)
    drop_element<T, RES>(x, res, y, i, d, seed);
}

template <class T, bool RES>
cudaError_t launch(const T* x, const T* res, int64_t n, const DropArgs& d, T* y, int num_sms,
                   cudaStream_t s) {
  const bool aligned16 = (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) |
                          reinterpret_cast<uintptr_t>(res)) % 16 == 0;
  const int64_t items = aligned16 ? (n >> 3) + 1 : n;  // + 1: the tail
  const int64_t per_block = kDropThreads * static_cast<int64_t>(aligned16 ? kDropGroups : 1);
  const int64_t blocks = (items + per_block - 1) / per_block;
  const int64_t most = static_cast<int64_t>(num_sms) * 8;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most)), block(kDropThreads);
  if (!aligned16) return launch_pdl(k_dropout_unaligned<T, RES>, grid, block, 0, s, x, res, n, d, y);
  if (d.offset & 1) return launch_pdl(k_dropout<T, RES, true>, grid, block, 0, s, x, res, n, d, y);
  return launch_pdl(k_dropout<T, RES, false>, grid, block, 0, s, x, res, n, d, y);
}

template <class T>
cudaError_t launch(const void* x, const void* res, int64_t n, const DropArgs& d, void* y,
                   int num_sms, cudaStream_t s) {
  const T* xt = static_cast<const T*>(x);
  return res ? launch<T, true>(xt, static_cast<const T*>(res), n, d, static_cast<T*>(y), num_sms, s)
             : launch<T, false>(xt, nullptr, n, d, static_cast<T*>(y), num_sms, s);
}

ss_status dropout_call(const void* x, const void* res, int64_t n, int dtype,
                       const ss_dropout_spec* drop, void* y, ss_stream stream, const char* name) {
  DropArgs d;
  if (n < 0 || (dtype != SS_BF16 && dtype != SS_FP32) || !make_drop_args(drop, &d))
    return SS_ERR_INVALID;
  if (n >= (int64_t(1) << 62)) return SS_ERR_UNSUPPORTED;
  if (n == 0) return SS_OK;
  const uintptr_t size = dtype == SS_BF16 ? 2 : 4;
  if (!x || !y || (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(res) |
                   reinterpret_cast<uintptr_t>(y)) % size != 0)
    return SS_ERR_INVALID;
  const int nsm = current_num_sms();
  if (nsm <= 0) return record_failure("cudaGetDevice/cudaDeviceGetAttribute", cudaGetLastError());
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  StageTrace trace(s, name);
  const cudaError_t e = dtype == SS_BF16 ? launch<uint16_t>(x, res, n, d, y, nsm, s)
                                         : launch<float>(x, res, n, d, y, nsm, s);
  return e == cudaSuccess ? SS_OK : record_failure(name, e);
}

}  // namespace

cudaError_t launch_drop_mask(const uint16_t* x, int64_t n, const DropArgs& drop, uint16_t* y,
                             int num_sms, cudaStream_t stream) {
  DropArgs d = drop;
  d.scale = 1.f;
  return launch<uint16_t, false>(x, nullptr, n, d, y, num_sms, stream);
}

}  // namespace ss

extern "C" {

ss_status ss_dropout(const void* x, const void* residual, int64_t n, int dtype,
                     const ss_dropout_spec* drop, void* y, ss_stream stream) {
  return ss::dropout_call(x, residual, n, dtype, drop, y, stream, "dropout");
}

ss_status ss_dropout_backward(const void* dy, int64_t n, int dtype, const ss_dropout_spec* drop,
                              void* dx, ss_stream stream) {
  return ss::dropout_call(dy, nullptr, n, dtype, drop, dx, stream, "dropout_backward");
}

}  // extern "C"
