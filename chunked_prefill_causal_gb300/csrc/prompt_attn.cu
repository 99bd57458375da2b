// prompt_attn.cu -- causal attention of whole prompts, packed one after the
// other, straight from the projection's q, k and v (no cache).
//
// "VPP: Virtual Pipeline Parallelism for Efficient Chunked Prefill in
// Long-Context LLM Inference" (technical review), §2.2, Eq. (1): token i of a
// sequence attends to that sequence's tokens <= i.
#include "ptx.cuh"
#include "serve.cuh"

namespace vpp {
namespace {

constexpr float kLn2q = 0.69314718055994530942f;

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// One warp per (token, head); a lane holds dims lane + 32 i.
__global__ void __launch_bounds__(128) prompt_kernel(const __grid_constant__ PromptParams p) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= p.total_q * p.heads) return;
  const int64_t t = w / p.heads;
  const int h = static_cast<int>(w % p.heads), g = h / (p.heads / p.kv_heads);
  const int b = find_seq(p.cu, p.batch, t);
  const int64_t lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1);
  if (w == 0 && lane == 0)
    for (int i = 0; i < p.batch; ++i)
      if (p.cu[i] < 0 || p.cu[i + 1] < p.cu[i] || p.cu[i + 1] > p.total_q) record_status(p.status, kStatusInvalid);
  if (lo < 0 || t < lo || t >= hi || hi > p.total_q) return;
  float q[6], o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < p.dq / 32; ++i) q[i] = bf(p.q[t * p.q_stride + h * p.dq + lane + 32 * i]);
  float m = -INFINITY, l = 0.f;
  for (int64_t j = lo; j <= t; ++j) {
    float s = 0.f;
    for (int i = 0; i < p.dq / 32; ++i) s += q[i] * bf(p.k[j * p.k_stride + g * p.dq + lane + 32 * i]);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), f = ex2_approx(m - mn), e = ex2_approx(s - mn);
    m = mn;
    l = l * f + e;
    for (int i = 0; i < p.dv / 32; ++i) o[i] = o[i] * f + e * bf(p.v[j * p.v_stride + g * p.dv + lane + 32 * i]);
  }
  for (int i = 0; i < p.dv / 32; ++i)
    p.out[(t * p.heads + h) * p.dv + lane + 32 * i] = static_cast<uint16_t>(pack_bf16x2(o[i] / l, 0.f) & 0xFFFF);
  if (p.lse && lane == 0) p.lse[h * p.total_q + t] = m * kLn2q + logf(l);
}

}  // namespace

size_t prompt_ws_bytes(int32_t, int64_t, int, int) { return 0; }

cudaError_t launch_prompt_attn(const PromptParams& p, void*, int, cudaStream_t stream) {
  prompt_kernel<<<static_cast<unsigned>((p.total_q * p.heads + 3) / 4), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vpp
