// serve.cuh -- parameters of the serving-step kernels whose lengths live on
// the device (rotate-and-append, decode attention),
// shared with api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace vpp {

// Rotate and append (rope_append.cu).  Strides are elements between tokens.
struct RopeParams {
  const uint16_t* q;         // bf16 [total_q][heads][dq], may be null
  const uint16_t* k;         // bf16 [total_q][kv_heads][dq]
  const uint16_t* v;         // bf16 [total_q][kv_heads][dv], unused without a cache
  uint16_t* q_out;
  uint16_t* k_out;           // may be null
  void* k_cache;             // [num_blocks][64][kv_heads][d], bf16 or E4M3 codes; null: no append
  void* v_cache;
  const float* k_scale;      // E4M3 cache: [kv_heads] factors (null for bf16)
  const float* v_scale;
  const float* cos_sin;      // [table_rows][rot_dim]: cosines, then sines
  const int32_t* block_table;
  const int32_t* cu;         // [batch + 1]
  const int32_t* ctx;        // [batch], null: every sequence's tokens are all of it
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int64_t total_q;
  int32_t batch;
  int32_t max_blocks_per_seq;
  int32_t num_blocks;
  int32_t table_rows;
  int32_t heads, kv_heads, dq, dv;
  int32_t rot_start, rot_dim;
  int* status;
};

cudaError_t launch_rope_append(const RopeParams& p, bool interleaved, bool fp8, int num_sms, cudaStream_t stream);

// Decode attention (decode_paged.cu).
struct PagedDecodeParams {
  const uint16_t* q;           // bf16 [batch][heads][dq], row stride q_stride
  const void* k_cache;         // [num_blocks][64][kv_heads][d], bf16 or E4M3 codes
  const void* v_cache;
  const float* k_scale;        // E4M3 cache: [kv_heads] factors (null for bf16)
  const float* v_scale;
  const int32_t* block_table;  // [batch][max_blocks_per_seq]
  const int32_t* ctx;          // [batch]
  uint16_t* out;               // bf16 [batch][heads][dv]
  float* lse;                  // [heads][batch], may be null
  int64_t q_stride;
  int32_t batch;
  int32_t max_blocks_per_seq;
  int32_t num_blocks;
  int32_t heads, kv_heads, dq, dv;
  float scale_log2;            // softmax scale * log2(e)
  int* status;
};

size_t paged_decode_ws_bytes(int32_t batch, int heads, int kv_heads, int dq, int dv, int num_sms);
// maps: K and V of the cache in boxes of 64 tokens, then in boxes of 16.
cudaError_t launch_paged_decode(const PagedDecodeParams& p, bool fp8, const CUtensorMap* maps, void* workspace,
                                int num_sms, cudaStream_t stream);

// The sequence that owns packed row t: the last b with cu[b] <= t (0 when
// there is none; the caller checks t against the sequence's range).
__device__ __forceinline__ int find_seq(const int32_t* cu, int32_t batch, int64_t t) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace vpp
