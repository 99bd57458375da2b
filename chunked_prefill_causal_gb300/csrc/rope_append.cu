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
//
// Bound by HBM for many tokens (each input is read and each output written
// once), by the latency of the chain lengths -> block and table row -> stores
// for few.  Measured on a GB300: 16384 tokens of 64 + 8 heads of 128, 679 MB,
// in 103.4 us (6.57 TB/s, 97% of the copy bandwidth); 4 decode tokens in 2.5 us.
// Into an E4M3 cache 646 MB in 113.5 us (84%), 4 decode tokens in 3.6 us: 16 quotients
// a task, and 60 bytes a thread spilled at 64 registers.
//
// Work split.  A row (one head of one token) is d / 16 tasks of two 16-byte
// vectors: eight pairs of the rotated dims (both ends of the pairs, so that one
// thread holds them whole and rotation in place is safe), or 16 copied values.
// A token is served by 64 threads of a CTA, or by all 256 when there are few
// tokens.  A thread keeps its task for every row of the token, so the eight
// cosines and sines are loaded once for all heads; two rows are in flight at
// once, the first ones while the token's position is looked up, and the angles load
// beside the block-table entry (one after the other: 2.8 us for the 4 tokens).
#include <algorithm>

#include "ptx.cuh"
#include "serve.cuh"

namespace vpp {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 4;  // CTAs per SM
constexpr int kMaxTile = 4;   // tokens of a CTA (a power of two)
constexpr int kRows = 2;      // rows in flight per thread
constexpr int kRopeWaves = 4;  // waves of CTAs to aim at

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 16 bytes that no other thread of the SM reads.  (Not the read-only path: with
// rotation in place this thread writes them afterwards.)
__device__ __forceinline__ uint4 ld_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf_lo(w.x); x[1] = bf_hi(w.x); x[2] = bf_lo(w.y); x[3] = bf_hi(w.y);
  x[4] = bf_lo(w.z); x[5] = bf_hi(w.z); x[6] = bf_lo(w.w); x[7] = bf_hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Eight E4M3 codes of x / scale (IEEE quotients).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_e4m3x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Where a token belongs: its sequence and its position there (-1: padding or invalid).
struct Place {
  int32_t b;
  int32_t pos;
};

__device__ __forceinline__ Place place_of(const RopeParams& p, int64_t t) {
  // A decode batch has one token per sequence: try sequence t first, its length
  // loaded beside its rows.
  int b = -1;
  int64_t lo = 0, hi = 0, ctx = 0;
  if (t < p.batch) {
    lo = __ldg(p.cu + t);
    hi = __ldg(p.cu + t + 1);
    if (p.ctx) ctx = __ldg(p.ctx + t);
    if (lo <= t && t < hi) b = static_cast<int>(t);
  }
  if (b < 0) {
    b = find_seq(p.cu, p.batch, t);
    lo = __ldg(p.cu + b);
    hi = __ldg(p.cu + b + 1);
    if (p.ctx) ctx = __ldg(p.ctx + b);
  }
  if (t < lo || t >= hi) return Place{0, -1};
  if (!p.ctx) ctx = hi - lo;
  if (ctx == 0) return Place{0, -1};
  const int64_t pos = ctx - (hi - t);
  if (ctx < hi - lo || pos < 0 || (p.rot_dim > 0 && pos >= p.table_rows) ||
      (p.k_cache && pos / kBlockTokens >= p.max_blocks_per_seq)) {
    record_status(p.status, kStatusInvalid);
    return Place{0, -1};
  }
  return Place{b, static_cast<int32_t>(pos)};
}

// Rotates the eight pairs of a task in float32.
template <bool IL>
__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const float (&cs)[8], const float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // pair e: (x_e, y_e), or interleaved (x_2e, x_2e+1) for e < 4, then y's
    float& u = !IL ? x[e] : e < 4 ? x[2 * e] : y[2 * e - 8];
    float& v = !IL ? y[e] : e < 4 ? x[2 * e + 1] : y[2 * e - 7];
    const float a = u, b = v;
    u = fmaf(a, cs[e], -__fmul_rn(b, sn[e]));
    v = fmaf(b, cs[e], __fmul_rn(a, sn[e]));
  }
}

template <bool IL, bool F8>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_append_kernel(const __grid_constant__ RopeParams p,
                                                                              const int tile) {
  grid_wait();
  // Thread i of the token's `wide` threads.
  const int wide = kRopeThreads / tile;
  const int i = threadIdx.x % wide;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * tile + threadIdx.x / wide;
  if (t >= p.total_q) return;

  // This thread's task of a query or key row: vectors at dims d0 and d1, and
  // the first of its eight angles (-1: copied).
  const int per = p.dq / 16;  // tasks of a row
  const int c = i % per, first = i / per, step = wide / per;
  const int rot = p.rot_dim / 16;
  int d0, d1, angle = -1;
  if (c < rot) {
    d0 = p.rot_start + (IL ? 16 * c : 8 * c);
    d1 = d0 + (IL ? 8 : p.rot_dim / 2);
    angle = 8 * c;
  } else {
    const int v = 2 * (c - rot), head = p.rot_start / 8;  // copied vectors v, v + 1
    d0 = 8 * v + (v < head ? 0 : p.rot_dim);
    d1 = 8 * (v + 1) + (v + 1 < head ? 0 : p.rot_dim);
  }
  const int hq = p.q ? p.heads : 0;
  // (threads past the last whole group of `per` have no row)
  const int rows = first < step ? hq + p.kv_heads : 0;
  const uint16_t* qs = p.q + t * p.q_stride;
  const uint16_t* ks = p.k + t * p.k_stride - static_cast<int64_t>(hq) * p.dq;
  uint4 a[kRows], b[kRows];
  float scales[kRows];
  auto load = [&](int r0) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = r0 + j * step;
      if (r < rows) {
        const uint16_t* src = (r < hq ? qs : ks) + r * p.dq;
        a[j] = ld_once(src + d0);
        b[j] = ld_once(src + d1);
        if (F8 && r >= hq) scales[j] = __ldg(p.k_scale + r - hq);
      }
    }
  };
  // gridDim.y CTAs share a token's rows, kRows passes at a time.
  const int begin = first + blockIdx.y * kRows * step, stride = gridDim.y * kRows * step;
  load(begin);  // in flight while the token's place is looked up

  if (t == 0 && i == 0 && blockIdx.y == 0 && __ldg(p.cu + p.batch) > p.total_q) record_status(p.status, kStatusInvalid);
  const Place at = place_of(p, t);
  if (at.pos < 0) return;
  // the angles load beside the block
  int32_t blk = 0;
  if (p.k_cache)
    blk = __ldg(p.block_table + static_cast<int64_t>(at.b) * p.max_blocks_per_seq + at.pos / kBlockTokens);
  float cs[8], sn[8];
  if (angle >= 0) {
    const float* src = p.cos_sin + static_cast<int64_t>(at.pos) * p.rot_dim + angle;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(src + e));
      const float4 y = __ldg(reinterpret_cast<const float4*>(src + p.rot_dim / 2 + e));
      cs[e] = x.x; cs[e + 1] = x.y; cs[e + 2] = x.z; cs[e + 3] = x.w;
      sn[e] = y.x; sn[e + 1] = y.y; sn[e + 2] = y.z; sn[e + 3] = y.w;
    }
  }
  if (p.k_cache && (blk < 0 || blk >= p.num_blocks)) {
    record_status(p.status, kStatusInvalid);
    return;
  }
  const int64_t slot = static_cast<int64_t>(blk) * kBlockTokens + at.pos % kBlockTokens;
  for (int r0 = begin; r0 < rows; r0 += stride) {
    if (r0 != begin) load(r0);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = r0 + j * step;
      if (r >= rows) continue;
      float x[8], y[8];
      if (angle >= 0 || F8) {
        unpack8(a[j], x);
        unpack8(b[j], y);
      }
      if (angle >= 0) {
        turn<IL>(x, y, cs, sn);
        a[j] = pack8(x);
        b[j] = pack8(y);
      }
      auto put = [&](uint16_t* dst) {
        *reinterpret_cast<uint4*>(dst + d0) = a[j];
        *reinterpret_cast<uint4*>(dst + d1) = b[j];
      };
      if (r < hq) {
        put(p.q_out + t * p.q_out_stride + r * p.dq);
      } else {
        const int h = r - hq;
        const int64_t row = (slot * p.kv_heads + h) * p.dq;
        if (p.k_out) put(p.k_out + t * p.k_out_stride + h * p.dq);
        if (F8) {
          const float scale = scales[j];
          uint8_t* dst = static_cast<uint8_t*>(p.k_cache) + row;
          *reinterpret_cast<uint2*>(dst + d0) = codes8(x, scale);
          *reinterpret_cast<uint2*>(dst + d1) = codes8(y, scale);
        } else if (p.k_cache) {
          put(static_cast<uint16_t*>(p.k_cache) + row);
        }
      }
    }
  }
  if (!p.k_cache) return;
  // values: the token's kv heads are contiguous on both sides
  const uint16_t* vs = p.v + t * p.v_stride;
  const int64_t row = slot * p.kv_heads * p.dv;
  const int n = p.kv_heads * p.dv / 8;
  for (int e0 = i + blockIdx.y * 2 * kRows * wide; e0 < n; e0 += gridDim.y * 2 * kRows * wide) {
    uint4 w[2 * kRows];
    float scale[2 * kRows];
#pragma unroll
    for (int j = 0; j < 2 * kRows; ++j)
      if (e0 + j * wide < n) {
        w[j] = ld_once(vs + 8 * (e0 + j * wide));
        if (F8) scale[j] = __ldg(p.v_scale + 8 * (e0 + j * wide) / p.dv);
      }
#pragma unroll
    for (int j = 0; j < 2 * kRows; ++j) {
      const int e = e0 + j * wide;
      if (e >= n) continue;
      if (F8) {
        float x[8];
        unpack8(w[j], x);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v_cache) + row + 8 * e) =
            codes8(x, scale[j]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_cache) + row + 8 * e) = w[j];
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, bool interleaved, bool fp8, int num_sms, cudaStream_t stream) {
  // One token a CTA until every SM has its CTAs, then up to kMaxTile.
  int tile = 1;
  while (tile < kMaxTile && p.total_q >= static_cast<int64_t>(2 * tile) * kRopeCtas * num_sms) tile *= 2;
  // Tokens of many rows are shared by several CTAs while there are fewer than
  // kRopeWaves waves of them: 800 tokens of 128 + 128 rows of 192 take 22.3 us with
  // one CTA a token and 21.5 us with several (256 decode tokens: 6.1 and 5.1 us).
  const int64_t ctas = (p.total_q + tile - 1) / tile;
  const int pass = kRows * (kRopeThreads / tile / (p.dq / 16));  // rows in flight
  const int passes = ((p.q ? p.heads : 0) + p.kv_heads + pass - 1) / pass;
  const int64_t want = (static_cast<int64_t>(kRopeWaves) * kRopeCtas * num_sms + ctas - 1) / ctas;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(passes, want))));
  const auto kernel = interleaved ? (fp8 ? rope_append_kernel<true, true> : rope_append_kernel<true, false>)
                                  : (fp8 ? rope_append_kernel<false, true> : rope_append_kernel<false, false>);
  return launch_overlapped(kernel, grid, kRopeThreads, 0, stream, p, tile);
}

}  // namespace vpp
