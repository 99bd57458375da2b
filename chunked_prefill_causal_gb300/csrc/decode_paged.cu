// decode_paged.cu -- attention of one new token per sequence over a paged KV
// cache, with the context lengths read on the device.
//
// "VPP: Virtual Pipeline Parallelism for Efficient Chunked Prefill in
// Long-Context LLM Inference" (technical review), §2.1 (decode reads the whole
// accumulated cache) and §2.2, Eq. (1), for a query at position ctx - 1:
//     out = sum_j exp(s_j - L) v_j,   s_j = scale q . k_j,   L = ln sum_j exp(s_j)
// over keys 0 .. ctx - 1, evaluated online (running max and denominator).
#include "ptx.cuh"
#include "serve.cuh"

namespace vpp {
namespace {

constexpr float kLn2p = 0.69314718055994530942f;

template <bool F8>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if (F8) {
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(static_cast<const uint8_t*>(p)[i], lo, hi);
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(lo));
    return f;
  }
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

// One warp per (row, head); a lane holds dims lane + 32 i.
template <bool F8>
__global__ void __launch_bounds__(128) paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(p.batch) * p.heads) return;
  const int b = static_cast<int>(w / p.heads), h = static_cast<int>(w % p.heads);
  const int g = h / (p.heads / p.kv_heads);
  int ctx = __ldg(p.ctx + b);
  if (ctx < 0 || ctx > static_cast<int64_t>(p.max_blocks_per_seq) * kBlockTokens) {
    if (lane == 0) record_status(p.status, kStatusInvalid);
    ctx = 0;
  }
  float q[6], o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < p.dq / 32; ++i)
    q[i] = __uint_as_float(static_cast<uint32_t>(p.q[b * p.q_stride + h * p.dq + lane + 32 * i]) << 16);
  const float sl = F8 ? p.scale_log2 * __ldg(p.k_scale + g) : p.scale_log2;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < ctx; ++j) {
    const int32_t blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq + j / kBlockTokens);
    const bool ok = blk >= 0 && blk < p.num_blocks;
    if (!ok && lane == 0) record_status(p.status, kStatusInvalid);
    const int64_t row = (static_cast<int64_t>(blk) * kBlockTokens + j % kBlockTokens) * p.kv_heads + g;
    float s = 0.f;
    for (int i = 0; i < p.dq / 32; ++i) s += ok ? q[i] * load_elem<F8>(p.k_cache, row * p.dq + lane + 32 * i) : 0.f;
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= sl;
    const float mn = fmaxf(m, s), f = ex2_approx(m - mn), e = ex2_approx(s - mn);
    m = mn;
    l = l * f + e;
    for (int i = 0; i < p.dv / 32; ++i)
      o[i] = o[i] * f + (ok ? e * load_elem<F8>(p.v_cache, row * p.dv + lane + 32 * i) : 0.f);
  }
  const float inv = l > 0.f ? (F8 ? __ldg(p.v_scale + g) : 1.f) / l : 0.f;
  for (int i = 0; i < p.dv / 32; ++i)
    p.out[(static_cast<int64_t>(b) * p.heads + h) * p.dv + lane + 32 * i] =
        static_cast<uint16_t>(pack_bf16x2(o[i] * inv, 0.f) & 0xFFFF);
  if (p.lse && lane == 0) p.lse[static_cast<int64_t>(h) * p.batch + b] = l > 0.f ? m * kLn2p + logf(l) : -INFINITY;
}

}  // namespace

size_t paged_decode_ws_bytes(int32_t, int, int, int, int, int) { return 0; }

cudaError_t launch_paged_decode(const PagedDecodeParams& p, bool fp8, void*, int, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(p.batch) * p.heads;
  const int grid = static_cast<int>((warps + 3) / 4);
  if (fp8)
    paged_decode_kernel<true><<<grid, 128, 0, stream>>>(p);
  else
    paged_decode_kernel<false><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vpp
