// ss_dropout.cu -- dropout and its gradient as one pass over the data:
//   y = residual + (kept ? scale * x : 0)
// The mask comes from ss_dropout.cuh and is stored nowhere.
//
// Groups of 8 elements keep every access 16 bytes wide. In fp32 and with a
// residual (6 bytes an element or more) memory bounds it. bf16 without a
// residual moves 4 bytes an element, next to about 11 integer instructions for
// the hash and its comparison: there the integer pipe is the busiest unit (79%
// of its cycles) and the two overlap imperfectly.
//   bf16 65536 x 768 with residual : 49.8 us, 6.1 TB/s
//   fp32 16411 x 1021              : 23.2 us, 5.8 TB/s
//   bf16 65536 x 2048              : 94.5 us, 5.7 TB/s (with p = 0, that is
//                                    without hashes, 88; a copy takes 81.8)
// Buffers off a 16-byte boundary, which views of a tensor can be, are walked one
// element and one hash at a time: 241 us for 37 at 65536 x 768 in bf16 (246 for 50
// with a residual), 237 for 66 in fp32.
// Tried and slower: two groups in flight per thread (more registers, fewer
// threads: 114 us), the next group's loads issued ahead of the hash (105 to
// 115), and the hash's shifts as high products on the other pipe (95 to 112).
#include <algorithm>

#include "ss_ffn.cuh"

namespace ss {

namespace {

// Threads per block: kDropSmall, a block per kDropSmall groups, where memory
// bounds the kernel and where there are few groups; kDropLarge, two resident
// blocks per SM that walk the data, where the integer pipe does (bf16 without a
// residual): 94.5 us against 110.4 at 65536 x 2048, where the small blocks' own
// setup takes issue slots, but 52.2 against 49.8 us with a residual.
constexpr int kDropSmall = 256, kDropLarge = 1024;

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
template <class T, bool RES, bool ODD, int THREADS>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS)
    k_dropout(const T* x, const T* res, int64_t n, const DropArgs d, T* y) {
  pdl_enter();
  const uint64_t seed = drop_seed(d);
  const int64_t n8 = n >> 3;
  const int64_t step = static_cast<int64_t>(gridDim.x) * THREADS;
  int64_t g = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x;
  if (g < (n & 7)) drop_element<T, RES>(x, res, y, (n8 << 3) + g, d, seed);
  for (; g < n8; g += step) {
    const int64_t at = g << 3;
    Vec8 a = load8(x + at), r;
    if (RES) r = load8(res + at);
    if (d.mode == kDropRandom) {
      for_kept<8, ODD>(seed, d.offset + static_cast<uint64_t>(at), d.thr, [&](int i, bool kept) {
        a.v[i] = drop_one<RES>(a.v[i], RES ? r.v[i] : 0.f, kept, d.scale);
      });
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        a.v[i] = drop_one<RES>(a.v[i], RES ? r.v[i] : 0.f, d.mode == kDropNone, d.scale);
    }
    store8(y + at, a);
  }
}

template <class T, bool RES>
__global__ void __launch_bounds__(kDropSmall)
    k_dropout_unaligned(const T* x, const T* res, int64_t n, const DropArgs d, T* y) {
  pdl_enter();
  const uint64_t seed = drop_seed(d);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kDropSmall;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kDropSmall + threadIdx.x; i < n; i += step)
    drop_element<T, RES>(x, res, y, i, d, seed);
}

template <class T, bool RES, int THREADS>
cudaError_t launch_aligned(const T* x, const T* res, int64_t n, const DropArgs& d, T* y,
                           int64_t blocks, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(blocks)), block(THREADS);
  return (d.offset & 1)
             ? launch_pdl(k_dropout<T, RES, true, THREADS>, grid, block, 0, s, x, res, n, d, y)
             : launch_pdl(k_dropout<T, RES, false, THREADS>, grid, block, 0, s, x, res, n, d, y);
}

template <class T, bool RES>
cudaError_t launch(const T* x, const T* res, int64_t n, const DropArgs& d, T* y, int num_sms,
                   cudaStream_t s) {
  constexpr int64_t kMostBlocks = (int64_t(1) << 31) - 1;  // more groups are walked
  const bool aligned16 = (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) |
                          reinterpret_cast<uintptr_t>(res)) % 16 == 0;
  const int64_t items = aligned16 ? (n >> 3) + ((n & 7) != 0) : n;
  const int64_t small = std::min((items + kDropSmall - 1) / kDropSmall, kMostBlocks);
  if (!aligned16)
    return launch_pdl(k_dropout_unaligned<T, RES>, dim3(static_cast<unsigned>(small)),
                      dim3(kDropSmall), 0, s, x, res, n, d, y);
  if constexpr (sizeof(T) == 2 && !RES) {
    const int64_t large = 2 * static_cast<int64_t>(num_sms);
    if (items >= large * kDropLarge) return launch_aligned<T, RES, kDropLarge>(x, res, n, d, y, large, s);
  }
  return launch_aligned<T, RES, kDropSmall>(x, res, n, d, y, small, s);
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
