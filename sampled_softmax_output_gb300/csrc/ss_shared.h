// ss_shared.h -- what ss_api.cu offers to the entry points of ss_block.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ss.h"

namespace ss {

// the workspace header's size; its first word is the status word
constexpr size_t kHeaderBytes = 1024;

// SM count of the current device, or <= 0 on failure
int current_num_sms();

// keeps the text for ss_last_error(); returns SS_ERR_CUDA
ss_status record_failure(const char* what, cudaError_t e);

// row-major bf16 [outer, inner], row_bytes between rows, in boxes of box_outer
// rows x box_inner elements (32 or 64: swizzled over the 64 or 128 bytes)
bool make_bf16_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                   uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer);

// One stage of the launch trace (ss_trace_begin), from construction to the end
// of the scope.
struct StageTrace {
  StageTrace(cudaStream_t s, const char* name);
  ~StageTrace();
  StageTrace(const StageTrace&) = delete;
  StageTrace& operator=(const StageTrace&) = delete;
  cudaStream_t s_;
};

}  // namespace ss
