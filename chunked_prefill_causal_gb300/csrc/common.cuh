// common.cuh -- types shared by the host launch code and the kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace vpp {

constexpr int kBlockTokens = 64;    // paged KV block ("02 · 并行策略与 PP 切分" note, §1)
constexpr int kMaxBatch = 1024;     // sequences per mixed micro-batch (plan passed by value)

// Per-sequence description of a varlen batch, passed to kernels by value.
struct VarlenPlan {
  int32_t batch;
  int32_t max_blocks_per_seq;       // row stride of the block table
  int32_t cu_q[kMaxBatch + 1];      // packed query/new-token row offsets
  int32_t ctx[kMaxBatch];           // total keys of each sequence (incl. new tokens)
};

// Launches a kernel that may be placed before the one before it in the stream has
// ended (programmatic dependent launch); the kernel calls grid_wait() before its
// first global access.  It is placed once every CTA of the one before has ended, or
// called grid_launch_next().  Only the decode kernel calls it, for its own join kernel: a
// kernel placed between the CTAs of another finds the SM's registers and shared memory
// in pieces, and CTAs that do not fit then run last, by themselves (decode over an E4M3
// cache, 471 MB, call after call: 106 us so, 76 us without; append and decode 103 and
// 82 us, 24 ragged prompts 110 and 107).
template <typename... A>
cudaError_t launch_overlapped(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                              const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Kernel launchers (defined in the .cu files, called from api.cu).
cudaError_t launch_kv_append(const void* k_new, const void* v_new, bool in_fp32, void* k_cache,
                             void* v_cache, const int32_t* block_table, int32_t num_blocks,
                             int64_t prefix_len, int64_t chunk_len, int kv_heads, int dq, int dv,
                             int* status, int num_sms, cudaStream_t stream);

cudaError_t launch_kv_append_varlen(const void* k_new, const void* v_new, void* k_cache,
                                    void* v_cache, const int32_t* block_table,
                                    const VarlenPlan& plan, int32_t num_blocks, int kv_heads,
                                    int dq, int dv, int* status, int num_sms,
                                    cudaStream_t stream);

cudaError_t launch_convert_f32_bf16(const float* in, uint16_t* out, int64_t n, int num_sms,
                                    cudaStream_t stream);

cudaError_t launch_wait_timeout_selftest(int timeout_us, int* status, cudaStream_t stream);

}  // namespace vpp
