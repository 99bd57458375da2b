// rope_append.cu -- rotates the new queries and keys by their positions and
// appends the new keys and values to a paged cache.
//
// "VPP: Virtual Pipeline Parallelism for Efficient Chunked Prefill in
// Long-Context LLM Inference" (technical review), §2.1: prefill fills the KV
// cache that later chunks and decode read; "02 · 并行策略与 PP 切分", §1: the
// cache is a pool of 64-token blocks.
//
// A token at cache position n turns the pair (x, y) of its query and key
// vectors by the angle of table row n:
//     x' = x cos - y sin,   y' = y cos + x sin,
// where the pairs of the rotated dims [s, s + r) are (i, i + r/2), or
// (2i, 2i + 1) when interleaved.  The other dims and the values are copied.
// The products are float32; a result is rounded once, to bf16 or to the code
// of an E4M3 cache.
#include "ptx.cuh"
#include "serve.cuh"

namespace vpp {
namespace {

__device__ __forceinline__ float bf16_f32(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// One thread per element pair or copied element, row by row.
template <bool IL, bool F8>
__global__ void __launch_bounds__(256) rope_append_kernel(const __grid_constant__ RopeParams p) {
  const int64_t t = blockIdx.x;
  if (t == 0 && threadIdx.x == 0 && __ldg(p.cu + p.batch) > p.total_q) record_status(p.status, kStatusInvalid);
  const int b = find_seq(p.cu, p.batch, t);
  const int64_t lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1);
  if (t < lo || t >= hi) return;
  const int64_t ctx = p.ctx ? __ldg(p.ctx + b) : hi - lo;
  if (ctx == 0) return;
  const int64_t pos = ctx - (hi - t);
  int64_t slot = 0;
  bool ok = ctx >= hi - lo && pos >= 0 && (p.rot_dim == 0 || pos < p.table_rows);
  if (ok && p.k_cache) {
    ok = pos / kBlockTokens < p.max_blocks_per_seq;
    if (ok) {
      const int32_t blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq + pos / kBlockTokens);
      ok = blk >= 0 && blk < p.num_blocks;
      slot = static_cast<int64_t>(blk) * kBlockTokens + pos % kBlockTokens;
    }
  }
  if (!ok) {
    if (threadIdx.x == 0) record_status(p.status, kStatusInvalid);
    return;
  }
  const float* cs = p.cos_sin + pos * p.rot_dim;
  const int half = p.rot_dim / 2;
  auto put = [&](void* cache, const float* scale, int64_t row, int h, int d, int i, float x) {
    const int64_t at = (row * p.kv_heads + h) * d + i;
    if (F8) {
      static_cast<uint8_t*>(cache)[at] = static_cast<uint8_t>(pack_e4m3x2(__fdiv_rn(x, __ldg(scale + h)), 0.f) & 0xFF);
    } else {
      static_cast<uint16_t*>(cache)[at] = static_cast<uint16_t>(pack_bf16x2(x, 0.f) & 0xFFFF);
    }
  };
  const int hq = p.q ? p.heads : 0;
  const int n = (hq + p.kv_heads) * p.dq;
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const int row = e / p.dq, i = e - row * p.dq;
    const bool is_q = row < hq;
    const uint16_t* src = is_q ? p.q + t * p.q_stride + row * p.dq : p.k + t * p.k_stride + (row - hq) * p.dq;
    const int j = i - p.rot_start;
    float x[2] = {bf16_f32(src[i]), 0.f};
    int at[2] = {i, i};
    int cnt = 1;
    if (j >= 0 && j < p.rot_dim) {
      if (IL ? (j & 1) : (j >= half)) continue;  // done by the pair's first thread
      at[1] = IL ? i + 1 : i + half;
      const int f = IL ? j >> 1 : j;
      const float c = cs[f], s = cs[half + f], a = x[0], y = bf16_f32(src[at[1]]);
      x[0] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(y, s));
      x[1] = __fadd_rn(__fmul_rn(y, c), __fmul_rn(a, s));
      cnt = 2;
    }
    for (int u = 0; u < cnt; ++u) {
      const uint16_t r = static_cast<uint16_t>(pack_bf16x2(x[u], 0.f) & 0xFFFF);
      if (is_q) {
        p.q_out[t * p.q_out_stride + row * p.dq + at[u]] = r;
      } else {
        if (p.k_out) p.k_out[t * p.k_out_stride + (row - hq) * p.dq + at[u]] = r;
        if (p.k_cache) put(p.k_cache, p.k_scale, slot, row - hq, p.dq, at[u], x[u]);
      }
    }
  }
  if (!p.k_cache) return;
  for (int e = threadIdx.x; e < p.kv_heads * p.dv; e += blockDim.x)
    put(p.v_cache, p.v_scale, slot, e / p.dv, p.dv, e % p.dv, bf16_f32(p.v[t * p.v_stride + e]));
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, bool interleaved, bool fp8, int, cudaStream_t stream) {
  const int grid = static_cast<int>(p.total_q);
  if (interleaved)
    fp8 ? rope_append_kernel<true, true><<<grid, 256, 0, stream>>>(p)
        : rope_append_kernel<true, false><<<grid, 256, 0, stream>>>(p);
  else
    fp8 ? rope_append_kernel<false, true><<<grid, 256, 0, stream>>>(p)
        : rope_append_kernel<false, false><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vpp
