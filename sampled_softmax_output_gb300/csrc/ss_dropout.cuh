// ss_dropout.cuh -- the dropout mask from a counter-based generator, made where
// it is needed: by the elementwise kernels of ss_dropout.cu and by the
// epilogue of the feed-forward block's down projection.
//
// Element e takes 32 bits of SplitMix64 output number e >> 1 (low half for
// even e, high half for odd), so one 64-bit hash serves two elements: with one
// hash per element the integer work, not the memory, would bound the kernels.
#pragma once

#include <stdint.h>

#include "ss_block.h"

namespace ss {

constexpr uint64_t kSplitMixGamma = 0x9E3779B97F4A7C15ull;

// SplitMix64's output function; output number k of the stream seeded with s
// is splitmix_out(s + (k + 1) * kSplitMixGamma).
__host__ __device__ __forceinline__ uint64_t splitmix_out(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

enum DropMode { kDropNone = 0, kDropRandom = 1, kDropAll = 2 };

// ss_dropout_spec as the kernels take it.
struct DropArgs {
  int mode;                  // DropMode: p = 0, in between, p = 1
  uint32_t thr;              // dropped where bits < thr
  float scale;               // 1 / (1 - p)
  uint64_t seed, offset;
  const uint64_t* seed_dev;  // nullable: added to seed on the device
};

// false: p outside [0, 1], or seed_dev misaligned
inline bool make_drop_args(const ss_dropout_spec* d, DropArgs* out) {
  *out = DropArgs{kDropNone, 0u, 1.f, 0, 0, nullptr};
  if (!d) return true;
  if (!(d->p >= 0.0 && d->p <= 1.0) || reinterpret_cast<uintptr_t>(d->seed_dev) % 8 != 0)
    return false;
  if (d->p == 0.0) return true;
  out->mode = d->p < 1.0 ? kDropRandom : kDropAll;
  if (d->p < 1.0) {
    out->thr = static_cast<uint32_t>(d->p * 4294967296.0);
    out->scale = static_cast<float>(1.0 / (1.0 - d->p));
  }
  out->seed = d->seed;
  out->offset = d->offset;
  out->seed_dev = d->seed_dev;
  return true;
}

__device__ __forceinline__ uint64_t drop_seed(const DropArgs& d) {
  return d.seed_dev ? d.seed + *d.seed_dev : d.seed;
}

// Runs fn(i, kept) for i = 0 .. N - 1 over the elements e0 .. e0 + N - 1 of the
// stream (N even): N / 2 hashes where e0 is even, one more where it is odd.
template <int N, bool ODD, class F>
__device__ __forceinline__ void for_kept(uint64_t seed, uint64_t e0, uint32_t thr, F&& fn) {
  static_assert(N % 2 == 0, "pairs");
  uint64_t state = seed + ((e0 >> 1) + 1) * kSplitMixGamma;
  uint64_t h = ODD ? splitmix_out(state) : 0;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if (ODD) {
      state += kSplitMixGamma;
      const uint64_t g = splitmix_out(state);
      fn(i, static_cast<uint32_t>(h >> 32) >= thr);
      fn(i + 1, static_cast<uint32_t>(g) >= thr);
      h = g;
    } else {
      h = splitmix_out(state);
      fn(i, static_cast<uint32_t>(h) >= thr);
      fn(i + 1, static_cast<uint32_t>(h >> 32) >= thr);
      state += kSplitMixGamma;
    }
  }
}

}  // namespace ss
