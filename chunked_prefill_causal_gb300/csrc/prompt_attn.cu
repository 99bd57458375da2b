// prompt_attn.cu -- causal attention of whole prompts, packed one after the
// other, straight from the projection's q, k and v (no cache): the packed form
// of the chunk-attention kernel (chunk_attn_impl.cuh, PK).
//
// "VPP: Virtual Pipeline Parallelism for Efficient Chunked Prefill in
// Long-Context LLM Inference" (technical review), §2.2, Eq. (1): token i of a
// sequence attends to that sequence's tokens <= i.
#include "chunk_attn_impl.cuh"

namespace vpp {

cudaError_t launch_packed_attn(int dq, int dv, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, const PackedParams& p, int grid, cudaStream_t stream) {
  if (dq == 64 && dv == 64) return launch_packed_attn_t<64, 64>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 64 && dv == 128) return launch_packed_attn_t<64, 128>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 128 && dv == 64) return launch_packed_attn_t<128, 64>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 128 && dv == 128) return launch_packed_attn_t<128, 128>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 192 && dv == 64) return launch_packed_attn_t<192, 64>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 192 && dv == 128) return launch_packed_attn_t<192, 128>(tm_q, tm_k, tm_v, p, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace vpp
