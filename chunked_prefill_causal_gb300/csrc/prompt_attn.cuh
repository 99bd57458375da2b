// prompt_attn.cuh -- parameters of the packed prompt-attention kernel (shared
// with api.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace vpp {

struct PromptParams {
  const int32_t* cu;   // [batch + 1]
  uint16_t* out;       // bf16 [total][heads][dv]
  float* lse;          // [heads][total], may be null
  int64_t total;       // packed rows
  int32_t batch;
  int32_t heads;
  int32_t kv_heads;
  float scale_log2;    // softmax scale * log2(e)
  int* status;
  // (set by the launcher) tokens of an item, and divisions by them and by kv_heads
  int32_t item_tokens, item_shift, head_shift;
  uint64_t item_mul, head_mul;
};

// Query rows of a tile: kTileM / G tokens of the G heads of a kv head.
cudaError_t launch_prompt_attn(int dq, int dv, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, const PromptParams& p, int num_sms, cudaStream_t stream);

}  // namespace vpp
