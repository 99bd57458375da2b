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
// for few.
//
// Work split.  A row (one head of one token) is d / 16 tasks of two 16-byte vectors:
// eight pairs of the rotated dims (both ends of the pairs, so that one thread
// holds them whole and rotation in place is safe), or 16 copied values.  A
// thread keeps its task for every row of a token, so the eight cosines and
// sines are loaded once for all heads, and four rows are in flight at once.
// A CTA takes a few consecutive tokens and looks up their positions and slots
// side by side, one thread a token, while the first rows load.
#include <algorithm>

#include "ptx.cuh"
#include "serve.cuh"

namespace vpp {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxTile = 4;  // tokens of a CTA
constexpr int kRows = 4;     // rows in flight per thread

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

// Where a token goes: its position (-1: padding or invalid) and cache row.
struct Place {
  int64_t row;
  int32_t pos;
};

__device__ __forceinline__ Place place_of(const RopeParams& p, int64_t t) {
  // A decode batch has one token per sequence: try sequence t first.
  int b = -1;
  int64_t lo = 0, hi = 0;
  if (t < p.batch) {
    lo = __ldg(p.cu + t);
    hi = __ldg(p.cu + t + 1);
    if (lo <= t && t < hi) b = static_cast<int>(t);
  }
  if (b < 0) {
    b = find_seq(p.cu, p.batch, t);
    lo = __ldg(p.cu + b);
    hi = __ldg(p.cu + b + 1);
  }
  if (t < lo || t >= hi) return Place{0, -1};
  const int64_t ctx = p.ctx ? __ldg(p.ctx + b) : hi - lo;
  if (ctx == 0) return Place{0, -1};
  const int64_t pos = ctx - (hi - t);
  bool ok = ctx >= hi - lo && pos >= 0 && (p.rot_dim == 0 || pos < p.table_rows);
  int64_t row = 0;
  if (ok && p.k_cache) {
    ok = pos / kBlockTokens < p.max_blocks_per_seq;
    if (ok) {
      const int32_t blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq + pos / kBlockTokens);
      ok = blk >= 0 && blk < p.num_blocks;
      row = static_cast<int64_t>(blk) * kBlockTokens + pos % kBlockTokens;
    }
  }
  if (!ok) {
    record_status(p.status, kStatusInvalid);
    return Place{0, -1};
  }
  return Place{row, static_cast<int32_t>(pos)};
}

template <bool IL, bool F8>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_append_kernel(const __grid_constant__ RopeParams p,
                                                                      const int tile) {
  __shared__ Place places[kMaxTile];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tile), p.total_q - t0));
  if (static_cast<int>(threadIdx.x) < nt) places[threadIdx.x] = place_of(p, t0 + threadIdx.x);
  if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.cu + p.batch) > p.total_q) record_status(p.status, kStatusInvalid);

  // This thread's task of a query or key row: vectors at dims d0 and d1, and
  // the first of its eight angles (-1: copied).
  const int per = p.dq / 16;  // tasks of a row
  const int c = threadIdx.x % per, first = threadIdx.x / per, step = kRopeThreads / per;
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
  const int rows = hq + p.kv_heads;
  __syncthreads();

  for (int i = 0; i < nt; ++i) {
    const Place at = places[i];
    if (at.pos < 0) continue;
    const int64_t t = t0 + i;
    float cs[8], sn[8];
    if (angle >= 0) {
      const float4* src = reinterpret_cast<const float4*>(p.cos_sin + static_cast<int64_t>(at.pos) * p.rot_dim + angle);
      const float4 c0 = __ldg(src), c1 = __ldg(src + 1);
      const float4* src2 = reinterpret_cast<const float4*>(p.cos_sin + static_cast<int64_t>(at.pos) * p.rot_dim +
                                                           p.rot_dim / 2 + angle);
      const float4 s0 = __ldg(src2), s1 = __ldg(src2 + 1);
      cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w; cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
      sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w; sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
    }
    const uint16_t* qs = p.q + t * p.q_stride;
    const uint16_t* ks = p.k + t * p.k_stride;
    // (threads past the last whole group of `per` have no task)
    for (int r0 = first; first < step && r0 < rows; r0 += kRows * step) {
      uint4 a[kRows], b[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int r = r0 + j * step;
        if (r < rows) {
          const uint16_t* src = r < hq ? qs + r * p.dq : ks + (r - hq) * p.dq;
          a[j] = ld_once(src + d0);
          b[j] = ld_once(src + d1);
        }
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int r = r0 + j * step;
        if (r >= rows) continue;
        float x[8], y[8];
        unpack8(a[j], x);
        unpack8(b[j], y);
        if (angle >= 0) {
          if (IL) {  // pairs (x0, x1), ..., (y6, y7)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float u = x[2 * e], v = x[2 * e + 1], w = y[2 * e], z = y[2 * e + 1];
              x[2 * e] = __fsub_rn(__fmul_rn(u, cs[e]), __fmul_rn(v, sn[e]));
              x[2 * e + 1] = __fadd_rn(__fmul_rn(v, cs[e]), __fmul_rn(u, sn[e]));
              y[2 * e] = __fsub_rn(__fmul_rn(w, cs[4 + e]), __fmul_rn(z, sn[4 + e]));
              y[2 * e + 1] = __fadd_rn(__fmul_rn(z, cs[4 + e]), __fmul_rn(w, sn[4 + e]));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float u = x[e], v = y[e];
              x[e] = __fsub_rn(__fmul_rn(u, cs[e]), __fmul_rn(v, sn[e]));
              y[e] = __fadd_rn(__fmul_rn(v, cs[e]), __fmul_rn(u, sn[e]));
            }
          }
        }
        if (r < hq) {
          uint16_t* dst = p.q_out + t * p.q_out_stride + r * p.dq;
          *reinterpret_cast<uint4*>(dst + d0) = pack8(x);
          *reinterpret_cast<uint4*>(dst + d1) = pack8(y);
        } else {
          const int h = r - hq;
          if (p.k_out || !F8) {
            const uint4 u = pack8(x), v = pack8(y);
            if (p.k_out) {
              uint16_t* dst = p.k_out + t * p.k_out_stride + h * p.dq;
              *reinterpret_cast<uint4*>(dst + d0) = u;
              *reinterpret_cast<uint4*>(dst + d1) = v;
            }
            if (!F8 && p.k_cache) {
              uint16_t* dst = static_cast<uint16_t*>(p.k_cache) + (at.row * p.kv_heads + h) * p.dq;
              *reinterpret_cast<uint4*>(dst + d0) = u;
              *reinterpret_cast<uint4*>(dst + d1) = v;
            }
          }
          if (F8) {
            const float scale = __ldg(p.k_scale + h);
            uint8_t* dst = static_cast<uint8_t*>(p.k_cache) + (at.row * p.kv_heads + h) * p.dq;
            *reinterpret_cast<uint2*>(dst + d0) = codes8(x, scale);
            *reinterpret_cast<uint2*>(dst + d1) = codes8(y, scale);
          }
        }
      }
    }
    if (!p.k_cache) continue;
    // values: the token's kv heads are contiguous on both sides
    const uint16_t* vs = p.v + t * p.v_stride;
    const int n = p.kv_heads * p.dv / 8;
    for (int e0 = threadIdx.x; e0 < n; e0 += kRows * kRopeThreads) {
      uint4 a[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (e0 + j * kRopeThreads < n) a[j] = ld_once(vs + 8 * (e0 + j * kRopeThreads));
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int e = e0 + j * kRopeThreads;
        if (e >= n) continue;
        const int64_t dst = at.row * p.kv_heads * p.dv + 8 * e;
        if (F8) {
          float x[8];
          unpack8(a[j], x);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v_cache) + dst) =
              codes8(x, __ldg(p.v_scale + 8 * e / p.dv));
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_cache) + dst) = a[j];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, bool interleaved, bool fp8, int num_sms, cudaStream_t stream) {
  // One token a CTA until every SM has its three CTAs, then up to kMaxTile.
  const int tile = static_cast<int>(std::min<int64_t>(kMaxTile, std::max<int64_t>(1, p.total_q / (3 * num_sms))));
  const int grid = static_cast<int>((p.total_q + tile - 1) / tile);
  if (interleaved)
    fp8 ? rope_append_kernel<true, true><<<grid, kRopeThreads, 0, stream>>>(p, tile)
        : rope_append_kernel<true, false><<<grid, kRopeThreads, 0, stream>>>(p, tile);
  else
    fp8 ? rope_append_kernel<false, true><<<grid, kRopeThreads, 0, stream>>>(p, tile)
        : rope_append_kernel<false, false><<<grid, kRopeThreads, 0, stream>>>(p, tile);
  return cudaGetLastError();
}

}  // namespace vpp
