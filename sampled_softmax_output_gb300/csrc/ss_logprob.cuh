// ss_logprob.cuh -- what the sources of the head's log-probabilities share: the
// problem as the launchers take it.
#pragma once

#include "ss_internal.h"
#include "ss_logprob.h"
#include "ss_ptx.cuh"
#include "ss_shared.h"

namespace ss {

struct LogprobArgs {
  const uint16_t *H, *W;
  int T, V, D;
  HeadCap head;
  float cap, tau;
  int* status;
  int num_sms;
};

// ---- ss_logprob_fwd.cu

// The ids [T, K] of each 32 tokens sorted by the 128 columns they fall into, `bins`
// = 2 ceil(V / 256) of them, for the kernel below.
cudaError_t launch_bin_ids(const LogprobArgs& p, const int32_t* ids, int K, int bins,
                           uint32_t* sorted, uint16_t* bin_ends, cudaStream_t s);
// part[c][t] = (n, s): the sum of exp(z) of row t over columns 128 c to 128 c + 127 is
// 2^n s, n an integer near its largest logit (so that no digit is lost in taking it off
// or in joining partials), c < bins; (-inf, 0) past the end. z: the logits of the
// sorted ids, place by place.
cudaError_t launch_logprob_partials(const LogprobArgs& p, int K, const uint32_t* sorted,
                                    const uint16_t* bin_ends, float2* part, float* z,
                                    cudaStream_t s);

// The same for a few tokens in one kernel, with partials of its own: how many there are
// (0: too many tokens for it), part [parts][T].
constexpr int kFewTokens = 2, kMostFewParts = 1024;
int logprob_few_parts(int64_t T, int64_t V, int num_sms);
cudaError_t launch_logprob_few(const LogprobArgs& p, int K, const int32_t* ids, int parts,
                               float2* part, float* z, cudaStream_t s);

// ---- ss_logprob_gemm.cu

// G[t, j] = bf16(coef[t] exp(z[t, j] - lse[t]) dz/ds), 0 where coef[t] = 0; but entry[t],
// bf16, where j is ids[t] (ids null: nowhere). G [T, ldG]
cudaError_t launch_logprob_g(const LogprobArgs& p, const float* coef, const float* lse,
                             const int32_t* ids, const uint32_t* entry, uint16_t* G, int64_t ldG,
                             cudaStream_t s);

// ---- ss_logprob_grads.cu

// dH[t] = rowfac[t] (G W)[t], dW (=|+=) *scale G^T Hs; null: a factor of 1. part:
// logprob_part_bytes, 32-byte aligned, for partial sums of dH.
size_t logprob_part_bytes(int64_t T, int64_t D);
cudaError_t launch_logprob_grads(const LogprobArgs& p, const uint16_t* G, int64_t ldG,
                                 const uint16_t* Hs, const float* rowfac, const float* scale,
                                 float* part, uint16_t* dH, void* dW, int dw_fp32, int accumulate,
                                 cudaStream_t s);

}  // namespace ss
