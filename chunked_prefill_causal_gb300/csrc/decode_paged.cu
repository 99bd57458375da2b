// decode_paged.cu -- attention of one new token per sequence over a paged KV
// cache, with the context lengths read on the device.
//
// "VPP: Virtual Pipeline Parallelism for Efficient Chunked Prefill in
// Long-Context LLM Inference" (technical review), §2.1 (decode reads the whole
// accumulated cache) and §2.2, Eq. (1), for a query at position ctx - 1:
//     out = sum_j exp(s_j - L) v_j,   s_j = scale q . k_j,   L = ln sum_j exp(s_j)
// over keys 0 .. ctx - 1, evaluated online (running max and denominator).
//
// Bound by HBM: every cached key and value is read once and used for the G
// query heads of its kv head only.  Measured on a GB300 (copy bandwidth 6.78 TB/s):
// 256 sequences of 1024 to 32768 tokens, 8 kv heads of 128, 16.6 GB in 2.26 to
// 2.36 ms (7.05 to 7.35 TB/s by machine); 200 over an E4M3 cache 6.8 TB/s; one of
// 131071 tokens, 537 MB, in 82 to 84 us (6.4 to 6.5 TB/s).  One of 1000 tokens takes
// 6.3 us, the latency of two launches and of lengths -> block table -> page -> softmax
// -> join.
//
// Work split.  The pages (64-token blocks) of all sequences, in order, form
// one list of N pages.  It is cut into `cols` equal parts whatever the
// lengths are; CTA (column c, kv head h) takes pages [c N / cols,
// (c + 1) N / cols) of head h.  cols x kv_heads fills the SMs (two or three CTAs each)
// in whole waves, so the launch shape needs no length and every CTA reads the
// same number of pages.  The CTAs of one column are neighbours in launch order and
// read the same blocks at the same time, head by head.  A sequence
// inside one column is finished there; one that crosses columns leaves a
// float32 partial (sum, reference, denominator) per column, which decode_join_kernel adds up
// ("02 · 并行策略与 PP 切分" note, §7).  A column has at most two such
// sequences, its first and its last.
//
// CTA (160 threads):
//   warp 4      producer: one TMA box of 64 tokens x 64 dims (128 codes) per
//               slab of a page's K and V into a ring of stages; the
//               last page of a sequence in boxes of 16 tokens, so that a short
//               sequence does not read 64 rows for a few.  It looks up the
//               block table 32 pages at a time.
//   warps 0-3   tokens 16 w .. 16 w + 15 of the page: S^T = K Q^T and O^T += V^T P^T
//               on the warp-level tensor cores (mma.sync m16n8k16, float32
//               accumulation).  The 16 rows are tokens, then dims, the 8 columns query
//               heads (a group of 9 to 16 takes two products).  K and V come by
//               ldmatrix from the swizzled stage, and P^T goes from the
//               accumulators of S^T to the operand in registers.  (With the heads
//               as the rows, half of them empty for 8 heads, an E4M3 cache read
//               15% slower.)  The decode products need a few per cent of even this
//               tensor path; tcgen05's 128-row tiles would be 1/8 to 1/128 full.
// The four warps' running results are joined through shared memory at the end
// of each sequence.
//
// E4M3 cache: the codes are widened exactly to f16 operands (every E4M3 value
// is an f16 value) after ldmatrix; q is scaled per head by a power of two into f16's
// range; k_scale joins the score scale and v_scale the result.
#include <algorithm>
#include <type_traits>

#include <cuda.h>

#include "ptx.cuh"
#include "serve.cuh"

namespace vpp {
namespace {

constexpr float kLn2p = 0.69314718055994530942f;
constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);

// A weight is 2^(score - m) for a reference m that is 2^kLift below the running maximum
// when it is taken and moves when the maximum has grown by more than 2^kGrow since (exact
// either way: numerator and denominator share it).  Over an E4M3 cache the weights
// become f16 operands, whose largest value is below 2^16: the largest weight lies in
// 2^14 .. 2^15, so a weight is rounded relatively (2^-11) down to 2^-28 of the largest one
// and absolutely (2^-39 of it) below.  (With the maximum itself as the reference, keys of
// 2^-25 of it and less were lost to the numerator, not to the denominator.)  bf16 operands
// have float32's range.
template <bool F8>
constexpr float kLift = F8 ? 14.0f : 0.0f;
template <bool F8>
constexpr float kGrow = F8 ? 1.0f : 8.0f;

// CTAs per SM: three where a stage is small and q and O take up to 80 registers of 128,
// else two.  (Two groups of heads over an E4M3 cache, 1.2 GB, two and three CTAs: 64/64
// dims 359 and 278 us, 64/128 277 and 264, 128/64 263 and 236, 192/64 229 and 207, the
// last three with 44, 12 and 112 bytes a thread spilled; 128/128, whose q and O take 96,
// 231 and 344.  Over a bf16 cache 64/64 dims take 178 and 182 us.)  192/128 dims with two
// groups spill 36 (bf16) and 64 bytes (E4M3) at two CTAs too.
constexpr int ctas_per_sm(int dq, int dv, bool f8, int ng) {
  return (ng == 1 || f8) && ng * (dq / 8 + dv / 4) <= 80 && (dq + dv) * (f8 ? 1 : 2) <= 256 ? 3 : 2;
}

// NG: query heads in groups of 8 (a kv head's G heads fill one or two).
template <int DQ, int DV, bool F8, int NG>
struct Cfg {
  static constexpr int ESZ = F8 ? 1 : 2;
  // Bytes of a slab row: 64 bf16 values, 128 codes (or 64 where the head dim
  // is no multiple of 128).
  static constexpr int KROW = F8 ? (DQ % 128 == 0 ? 128 : 64) : 128;
  static constexpr int VROW = F8 ? (DV % 128 == 0 ? 128 : 64) : 128;
  static constexpr int KSLABS = DQ * ESZ / KROW;
  static constexpr int VSLABS = DV * ESZ / VROW;
  static constexpr int KBYTES = DQ * ESZ * kBlockTokens;
  static constexpr int STAGE = KBYTES + DV * ESZ * kBlockTokens;
  static constexpr int CTAS = ctas_per_sm(DQ, DV, F8, NG);
  static constexpr int FIT = ((CTAS == 3 ? 56 : 96) * 1024) / STAGE;
  static constexpr int NST = FIT > 8 ? 8 : FIT;
  static constexpr int KS = DQ / 16;  // 16-dim steps of S^T
  static constexpr int NT = DV / 16;  // 16-dim tiles of O^T
  static constexpr int CSTRIDE = DV + 4;  // row stride of the join buffer: no two lanes of a store on a bank
  static constexpr int COMB = kConsumers * 8 * CSTRIDE * 4;
  static constexpr int SMEM = NST * STAGE + COMB + kConsumers * 8 * 8 + 2 * NST * 8 + 48;
  static_assert(NST >= 2, "two stages at least");
  static_assert(SMEM + 1024 <= 228 * 1024 / CTAS, "CTAs per SM");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// D (16 x 8, f32) += A (16 x 16) B (16 x 8), f16 or bf16 operands.
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Byte offset of 16-byte chunk c of row r in a slab that TMA wrote with the
// swizzle of its row width (128 or 64 bytes).
template <int ROW>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return ROW == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Transposes an 8x8 matrix of 16-bit values held one row pair per lane
// (lane 4 r + c: row r, columns 2c and 2c + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One thing the join kernel adds up: the parts of sequence b in columns
// c - 1 (slot `slot`) and c .. c + n - 2 (slot 0), filed under column c.
struct JoinDesc {
  int32_t b;  // -1: none
  int32_t n;
  int32_t slot;
  int32_t pad;
};

struct Workspace {
  float* o;      // [cols][2][heads][dv], sums relative to 2^reference
  float2* ml;    // [cols][2][heads], (reference, denominator)
  JoinDesc* desc;  // [cols]
};

// A context length as the kernels use it: 0 for one that does not fit its
// block-table row.
__device__ __forceinline__ int valid_ctx(const PagedDecodeParams& p, int ctx) {
  return (ctx < 0 || ctx > p.max_blocks_per_seq * kBlockTokens) ? 0 : ctx;
}
__device__ __forceinline__ int pages_of(int ctx) { return (ctx + kBlockTokens - 1) / kBlockTokens; }

// First page of column c: c total / nc, in 32 bits.
__device__ __forceinline__ int first_page(uint32_t c, uint32_t total, uint32_t nc) {
  const uint32_t share = total / nc, extra = total - share * nc;
  return static_cast<int>(c * share + c * extra / nc);
}

// Walks the non-empty sequences from one on; every lane of the warp holds one
// of 32 lengths, so a run of empty rows costs one load per 32.
struct SeqWalk {
  int base;  // first sequence of the lanes
  int mine;  // this lane's length
  int b;     // current sequence
  int ctx;
  __device__ __forceinline__ void load(const PagedDecodeParams& p, int from) {
    base = from;
    const int i = from + (threadIdx.x & 31);
    mine = i < p.batch ? valid_ctx(p, __ldg(p.ctx + i)) : 0;
  }
  // From sequence `at` on; `few` are the lengths of the first 32 where there are no more.
  __device__ __forceinline__ void start(const PagedDecodeParams& p, int at, int few) {
    if (p.batch <= 32) {
      base = 0;
      mine = few;
    } else {
      load(p, at);
    }
    b = at;
    ctx = __shfl_sync(0xffffffffu, mine, at - base);
  }
  // Goes on to the next non-empty sequence (there is one).
  __device__ __forceinline__ void next(const PagedDecodeParams& p) {
    int from = b - base + 1;
    while (true) {
      const uint32_t live = from < 32 ? __ballot_sync(0xffffffffu, mine > 0) & (0xffffffffu << from) : 0u;
      if (live) {
        const int l = __ffs(live) - 1;
        b = base + l;
        ctx = __shfl_sync(0xffffffffu, mine, l);
        return;
      }
      if (base + 32 >= p.batch) return;  // not reached while pages are left
      load(p, base + 32);
      from = 0;
    }
  }
};

template <int DQ, int DV, bool F8, int NG>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(DQ, DV, F8, NG))
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v16,
                        const __grid_constant__ PagedDecodeParams p, const Workspace ws, const int cols) {
  using C = Cfg<DQ, DV, F8, NG>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* comb = reinterpret_cast<float*>(smem + C::NST * C::STAGE);                  // [4][8][CSTRIDE]
  float2* ml = reinterpret_cast<float2*>(smem + C::NST * C::STAGE + C::COMB);        // [4][8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ml + kConsumers * 8);                 // full[NST], empty[NST]
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(bars + 2 * C::NST);
  int* scan = reinterpret_cast<int*>(const_cast<uint32_t*>(abort_flag) + 1);         // 5 sums, then (b, page)
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int col = blockIdx.x / p.kv_heads;
  const int h = blockIdx.x - col * p.kv_heads;
  const int G = p.heads / p.kv_heads;

  if (cols > 1) grid_launch_next();  // the join kernel may be placed beside this one

  if (threadIdx.x == 0) *abort_flag = 0u;
  if (threadIdx.x < 2 * C::NST) {
    mbar_init(smem_u32(&bars[threadIdx.x]), threadIdx.x < C::NST ? 1 : kConsumers);
    fence_mbar_init();
  }
  if (warp == kConsumers && lane < 4)
    tma_prefetch_desc(lane == 0 ? &tm_k : lane == 1 ? &tm_v : lane == 2 ? &tm_k16 : &tm_v16);
  grid_wait();
  // ---- this column's pages
  int total, nc, first, last, start_b = 0, start_page = 0;  // start_page: pages of start_b before this column
  int few = 0;  // this lane's length, where there are up to 32
  auto share_out = [&]() {
    nc = min(cols, total);  // columns with pages: at least one page each
    first = col < nc ? first_page(col, total, nc) : 0;
    last = col < nc ? first_page(col + 1, total, nc) : 0;  // one past
  };
  auto length_at = [&](int b, int end) {  // (an invalid length counts as 0 and is recorded)
    if (b >= end) return 0;
    const int raw = __ldg(p.ctx + b), c = valid_ctx(p, raw);
    if (c != raw && blockIdx.x == 0) record_status(p.status, kStatusInvalid);
    return c;
  };
  // Looks for the page `first` in the lanes' sequences, from `from` on, with `at` pages
  // before them.
  auto locate = [&](int from, int n, int inc, int at) {
    const uint32_t hit = __ballot_sync(0xffffffffu, first < at + inc);
    if (!hit) return false;
    const int l = __ffs(hit) - 1;
    start_b = from + l;
    start_page = first - __shfl_sync(0xffffffffu, at + inc - n, l);
    return true;
  };
  auto prefix = [&](int n) {  // inclusive, over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += y;
    }
    return n;
  };
  if (p.batch <= 32) {
    // every warp finds it by itself (one row of 1000 keys 6.8 -> 6.3 us)
    few = length_at(lane, p.batch);
    const int n = pages_of(few), inc = prefix(n);
    total = __shfl_sync(0xffffffffu, inc, 31);
    share_out();
    if (first < last) locate(0, n, inc, 0);
    __syncthreads();  // the barriers are set up
  } else {
    // warp w adds up the w-th fifth of the sequences, and the one whose range holds
    // the column's first page finds it
    const int per = (p.batch + 4) / 5;
    const int b0 = min(p.batch, warp * per), b1 = min(p.batch, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; b += 32) sum += pages_of(length_at(b + lane, b1));
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) scan[warp] = sum;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < 5; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    share_out();
    __syncthreads();
    if (first < last && first >= before && first < before + sum) {
      int at = before;
      for (int b = b0;; b += 32) {
        const int n = b + lane < b1 ? pages_of(valid_ctx(p, __ldg(p.ctx + b + lane))) : 0;
        const int inc = prefix(n);
        if (locate(b, n, inc, at)) break;
        at += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) {
        scan[5] = start_b;
        scan[6] = start_page;
      }
    }
    __syncthreads();
    if (first < last) {
      start_b = scan[5];
      start_page = scan[6];
    }
  }
  const int n_pages = last - first;

  if (warp == kConsumers) {
    // ------------------------------------------------------ producer
    if (n_pages > 0) {
      // The first 32 entries of the block table load while the sequence's length does.
      const int32_t* row = p.block_table + static_cast<int64_t>(start_b) * p.max_blocks_per_seq + start_page;
      int32_t next_blk = lane < p.max_blocks_per_seq - start_page ? __ldg(row + lane) : 0;
      // Starts the copies of a page with `rest` tokens of its sequence left.
      auto copy_page = [&](int slot, int32_t blk, int rest) {
        const uint32_t full = smem_u32(&bars[slot]);
        const uint32_t dk = smem_u32(smem + slot * C::STAGE), dv = dk + C::KBYTES;
        if (rest > kBlockTokens - 16) {
          mbar_arrive_expect_tx(full, C::STAGE);
#pragma unroll
          for (int s = 0; s < C::KSLABS; ++s)
            tma_load_4d(dk + s * C::KROW * kBlockTokens, &tm_k, full, s * (C::KROW / C::ESZ), h, 0, blk);
#pragma unroll
          for (int s = 0; s < C::VSLABS; ++s)
            tma_load_4d(dv + s * C::VROW * kBlockTokens, &tm_v, full, s * (C::VROW / C::ESZ), h, 0, blk);
        } else {
          const int groups = (rest + 15) / 16;
          mbar_arrive_expect_tx(full, groups * (C::STAGE / 4));
          for (int g = 0; g < groups; ++g) {
            for (int s = 0; s < C::KSLABS; ++s)
              tma_load_4d(dk + (s * kBlockTokens + 16 * g) * C::KROW, &tm_k16, full, s * (C::KROW / C::ESZ), h,
                          16 * g, blk);
            for (int s = 0; s < C::VSLABS; ++s)
              tma_load_4d(dv + (s * kBlockTokens + 16 * g) * C::VROW, &tm_v16, full, s * (C::VROW / C::ESZ), h,
                          16 * g, blk);
          }
        }
      };
      SeqWalk sw;
      sw.start(p, start_b, few);
      int page = start_page, left = n_pages;
      int slot = 0;
      uint32_t phase = 0u, filled = 0u, fill_phase = 0u;
      bool ok = true;
      while (ok && left > 0) {
        const int np = min(pages_of(sw.ctx) - page, left);
        for (int i = 0; ok && i < np; i += 32) {
          const int32_t blks = next_blk;  // lane l: block of page i + l
          // the next 32 entries load while these pages are copied
          next_blk = i + 32 + lane < np ? __ldg(row + i + 32 + lane) : 0;
          const int live = min(32, np - i);
          for (int j = 0; j < live; ++j) {
            int32_t blk = __shfl_sync(0xffffffffu, blks, j);
            if (blk < 0 || blk >= p.num_blocks) {
              if (lane == 0) record_status(p.status, kStatusInvalid);
              blk = p.num_blocks;  // out of the map: reads zeros
            }
            if (lane == 0) {
              ok = mbar_wait(smem_u32(&bars[C::NST + slot]), phase ^ 1u, p.status, abort_flag);
              if (ok) copy_page(slot, blk, sw.ctx - (page + i + j) * kBlockTokens);
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            filled |= 1u << slot;
            fill_phase = (fill_phase & ~(1u << slot)) | (phase << slot);
            if (++slot == C::NST) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
        left -= np;
        page = 0;
        if (left > 0) {
          sw.next(p);
          row = p.block_table + static_cast<int64_t>(sw.b) * p.max_blocks_per_seq;
          next_blk = lane < min(pages_of(sw.ctx), left) ? __ldg(row + lane) : 0;
        }
      }
      if (!ok && lane == 0) {
        // Let every copy land before the CTA exits.
        for (int i = 0; i < C::NST; ++i)
          if (filled & (1u << i)) mbar_wait_for(smem_u32(&bars[i]), (fill_phase >> i) & 1u, 100000000ull);
      }
    }
    if (h == 0 && lane == 0) {
      // File the sequence that column col - 1 ends with and this one goes on
      // with, if it began there: the parts of one sequence are one entry.
      JoinDesc d{-1, 0, 0, 0};
      if (n_pages > 0 && start_page > 0) {
        const int begin = first - start_page;  // the sequence's first page
        const int prev = first_page(col - 1, total, nc);
        if (begin >= prev) {
          const int64_t end = begin + pages_of(valid_ctx(p, __ldg(p.ctx + start_b)));  // one past
          const int last_col = static_cast<int>((end * nc - 1) / total);
          d = JoinDesc{start_b, last_col - col + 2, begin == prev ? 0 : 1, 0};
        }
      }
      if (cols > 1) ws.desc[col] = d;
    }
    return;
  }

  // -------------------------------------------------------- consumers
  // Rows of length 0: zeros, and -inf for the log of an empty sum.
  for (int b = col; b < p.batch; b += cols) {
    if ((p.batch <= 32 ? __shfl_sync(0xffffffffu, few, b) : valid_ctx(p, __ldg(p.ctx + b))) > 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(b) * p.heads + h * G) * DV);
    for (int i = threadIdx.x; i < G * DV / 8; i += 32 * kConsumers) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse && threadIdx.x < G) p.lse[static_cast<int64_t>(h * G + threadIdx.x) * p.batch + b] = -INFINITY;
  }
  if (n_pages == 0) return;

  const int g = lane >> 2, u = lane & 3;  // fragment row and column pair
  const int mi = lane >> 3, r8 = lane & 7;  // matrix and row that this lane addresses in ldmatrix
  const float sl = F8 ? p.scale_log2 * __ldg(p.k_scale + h) : p.scale_log2;
  const float vsc = F8 ? __ldg(p.v_scale + h) : 1.f;
  const uint32_t ring = smem_u32(smem);
  // Rows and chunks of this lane's ldmatrix addresses.  K (and V's codes): token halves,
  // then chunks; V: chunks, then token halves.
  const int krow = warp * 16 + (mi & 1) * 8 + r8, kchunk = mi >> 1;
  const int vrow = F8 ? krow : warp * 16 + (mi >> 1) * 8 + r8, vchunk = F8 ? kchunk : mi & 1;

  SeqWalk sw;
  sw.start(p, start_b, few);
  int page = start_page, left = n_pages;
  int slot = 0;
  uint32_t phase = 0u;
  bool ok = true;
  // q of a sequence as the B operand: column g is head g of the group (zeros
  // past G).  E4M3 cache: dims 4u .. 4u + 3 of a 16-dim step are a lane's (see
  // the K operand).
  uint32_t qb[NG][C::KS][2];
  float rs[NG][2];  // score scale of this thread's columns, heads 2u and 2u + 1
  auto load_q = [&](int b) {
    const uint16_t* qrow = p.q + b * p.q_stride + static_cast<int64_t>(h) * G * DQ;
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const bool live = 8 * n + g < G;
      const uint16_t* src = qrow + (live ? 8 * n + g : 0) * DQ;
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        uint2 w;
        if (F8) {
          w = __ldg(reinterpret_cast<const uint2*>(src + 16 * s + 4 * u));
        } else {
          w.x = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * u));
          w.y = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * u + 8));
        }
        qb[n][s][0] = live ? w.x : 0u;
        qb[n][s][1] = live ? w.y : 0u;
      }
      rs[n][0] = rs[n][1] = sl;
    }
  };
  // E4M3 cache: bf16 -> f16 in place, a head scaled by 2^e so that its largest
  // |q| is in [2^14, 2^15): below f16's largest value, and every bf16 value that
  // is not negligible beside it keeps its 8 significant bits.
  auto scale_q = [&]() {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      float amax = 0.f;
#pragma unroll
      for (int s = 0; s < C::KS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(qb[n][s][i])), fabsf(bf16_hi(qb[n][s][i]))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // (-113 at least; 126 at most, so that 2^e is a float32: reached below 2^-112)
      const int e = (amax > 0.f && amax < INFINITY) ? min(126, 14 - ilogbf(amax)) : 0;
      const float up = ldexpf(1.f, e), down = sl * ldexpf(1.f, -e);
      rs[n][0] = __shfl_sync(0xffffffffu, down, 8 * u);  // lane 4 (2u) holds head 2u
      rs[n][1] = __shfl_sync(0xffffffffu, down, 8 * u + 4);
#pragma unroll
      for (int s = 0; s < C::KS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qb[n][s][i] = pack_half2(bf16_lo(qb[n][s][i]) * up, bf16_hi(qb[n][s][i]) * up);
    }
  };
  load_q(start_b);
  while (left > 0) {
    const int seq_pages = pages_of(sw.ctx);
    const int np = min(seq_pages - page, left);
    if (F8) scale_q();
    float m[NG][2], l[NG][2];  // references of the weights, and this lane's part of the denominators
    float o[NG][C::NT][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int t = 0; t < C::NT; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
    }

    // 16 tokens of a stage, `live` of them keys of the sequence (all, unless TAIL).
    auto step = [&](auto tail, uint32_t kb, int live) {
      constexpr bool TAIL = decltype(tail)::value;
      const uint32_t vb = kb + C::KBYTES;
      // ---- S^T = K Q^T, 16 tokens x 8 heads; two accumulator chains
      float s[NG][2][4];
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) s[n][c][0] = s[n][c][1] = s[n][c][2] = s[n][c][3] = 0.f;
      if (!F8) {
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
          uint32_t r[4];
          ldsm4(kb + (k >> 2) * 128 * kBlockTokens + swz<128>(krow, 2 * (k & 3) + kchunk), r);
#pragma unroll
          for (int n = 0; n < NG; ++n) mma<false>(s[n][k & 1], r, qb[n][k][0], qb[n][k][1]);
        }
      } else {
        constexpr int CPS = C::KROW / 16;  // 16-code chunks of a slab row
#pragma unroll
        for (int k = 0; k < C::KS; k += 2) {
          uint32_t r[4];
          ldsm4(kb + (k / CPS) * C::KROW * kBlockTokens + swz<C::KROW>(krow, k % CPS + kchunk), r);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t a[4];
            e4m3x4_to_f16x2x2(r[2 * x], a[0], a[2]);
            e4m3x4_to_f16x2x2(r[2 * x + 1], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NG; ++n) mma<true>(s[n][x], a, qb[n][k + x][0], qb[n][k + x][1]);
          }
        }
      }
      uint32_t pb[NG][2];  // P^T as the B operand
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        // ---- scores in log2 units: [e >> 1: token g or g + 8][e & 1: head];
        // keys past the sequence leave the softmax
        float sc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[e] = (s[n][0][e] + s[n][1][e]) * rs[n][e & 1];
          if (TAIL && g + 8 * (e >> 1) >= live) sc[e] = -INFINITY;
        }
        // ---- online softmax of the two heads (eight lanes hold a head)
        float f[2];
        bool moved = false;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(sc[c], sc[2 + c]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          f[c] = 1.f;
          if (mx > m[n][c] + (kLift<F8> + kGrow<F8>) || (m[n][c] == -INFINITY && mx > -INFINITY)) {
            const float to = mx - kLift<F8>;
            f[c] = ex2_approx(m[n][c] - to);
            m[n][c] = to;
            moved = true;
          }
        }
        if (__any_sync(0xffffffffu, moved)) {
          l[n][0] *= f[0];
          l[n][1] *= f[1];
#pragma unroll
          for (int t = 0; t < C::NT; ++t) {
            o[n][t][0] *= f[0];
            o[n][t][1] *= f[1];
            o[n][t][2] *= f[0];
            o[n][t][3] *= f[1];
          }
        }
        float pv[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float mr = m[n][c] == -INFINITY ? 0.f : m[n][c];
          pv[c] = ex2_approx(sc[c] - mr);
          pv[2 + c] = ex2_approx(sc[2 + c] - mr);
          l[n][c] += pv[c] + pv[2 + c];
        }
        // P is rounded to the operand type of V (bf16, relative 2^-8; f16 over an
        // E4M3 cache, see kLift); the denominator keeps float32.
        // Its accumulator fragment, transposed, is the operand's.
        pb[n][0] = transpose8x8(F8 ? pack_half2(pv[0], pv[1]) : pack_bf16x2(pv[0], pv[1]));
        pb[n][1] = transpose8x8(F8 ? pack_half2(pv[2], pv[3]) : pack_bf16x2(pv[2], pv[3]));
      }
      // ---- O^T += V^T P^T.  Rows past the sequence may hold anything, and P = 0
      // times them must stay 0: their halves of the operand words are cleared.
      uint32_t mask[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      if (TAIL) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int at = 8 * t + 2 * u;
          mask[t] = (at < live ? 0x0000FFFFu : 0u) | (at + 1 < live ? 0xFFFF0000u : 0u);
        }
      }
      if (!F8) {
#pragma unroll
        for (int t = 0; t < C::NT; ++t) {
          uint32_t r[4];
          ldsm4_t(vb + (t >> 2) * 128 * kBlockTokens + swz<128>(vrow, 2 * (t & 3) + vchunk), r);
          if (TAIL) {
            r[0] &= mask[0];
            r[1] &= mask[0];
            r[2] &= mask[1];
            r[3] &= mask[1];
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) mma<false>(o[n][t], r, pb[n][0], pb[n][1]);
        }
      } else {
        // A word holds dims 2g, 2g + 1 of tokens 2u, 2u + 1: row g of the tile is
        // dim 2g of a 16-dim chunk, row g + 8 dim 2g + 1.
        constexpr int CPS = C::VROW / 16;
#pragma unroll
        for (int t = 0; t < C::NT; t += 2) {
          uint32_t r[4];
          ldsm4_t(vb + (t / CPS) * C::VROW * kBlockTokens + swz<C::VROW>(vrow, t % CPS + vchunk), r);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t a[4];
            if (TAIL) {
              r[2 * x] &= mask[0];
              r[2 * x + 1] &= mask[1];
            }
            e4m3x4_to_f16x2x2(__byte_perm(r[2 * x], 0u, 0x3120u), a[0], a[1]);
            e4m3x4_to_f16x2x2(__byte_perm(r[2 * x + 1], 0u, 0x3120u), a[2], a[3]);
#pragma unroll
            for (int n = 0; n < NG; ++n) mma<true>(o[n][t + x], a, pb[n][0], pb[n][1]);
          }
        }
      }
    };

    for (int i = 0; i < np; ++i) {
      // tokens of this warp's 16 that are keys of the sequence
      const int live = sw.ctx - (page + i) * kBlockTokens - warp * 16;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[slot]), phase, p.status, abort_flag));
      if (ok) {
        if (live >= 16)
          step(std::false_type{}, ring + slot * C::STAGE, 16);
        else if (live > 0)
          step(std::true_type{}, ring + slot * C::STAGE, live);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars[C::NST + slot]));
      if (++slot == C::NST) {
        slot = 0;
        phase ^= 1u;
      }
    }

    // The next sequence's q loads while this one's warps are joined.
    SeqWalk nx = sw;
    if (left > np) {
      nx.next(p);
      load_q(nx.b);
    }
    // ---- join the four warps, 8 rows at a time.  Every warp comes here for
    // every sequence, also after a failed wait, so the barriers match.
    const bool whole = np == seq_pages;
    const int part = (col * 2 + (page == start_page && left == n_pages ? 0 : 1));
#pragma unroll
    for (int half = 0; half < NG; ++half) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float lr = l[half][c];
        lr += __shfl_xor_sync(0xffffffffu, lr, 4);
        lr += __shfl_xor_sync(0xffffffffu, lr, 8);
        lr += __shfl_xor_sync(0xffffffffu, lr, 16);
        if (g == 0) ml[warp * 8 + 2 * u + c] = make_float2(m[half][c], lr);
        float* dst = comb + (warp * 8 + 2 * u + c) * C::CSTRIDE;
#pragma unroll
        for (int t = 0; t < C::NT; ++t) {
          if (!F8) {
            dst[16 * t + g] = o[half][t][c];
            dst[16 * t + 8 + g] = o[half][t][2 + c];
          } else {
            *reinterpret_cast<float2*>(dst + 16 * t + 2 * g) = make_float2(o[half][t][c], o[half][t][2 + c]);
          }
        }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      constexpr int PER = DV / 16;  // dims of a thread: 16 threads a row
      const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * PER;
      if (r + 8 * half < G) {
        float wgt[kConsumers], top = -INFINITY, den = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) top = fmaxf(top, ml[w * 8 + r].x);
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
          const float2 x = ml[w * 8 + r];
          wgt[w] = x.x == -INFINITY ? 0.f : ex2_approx(x.x - top);
          den += wgt[w] * x.y;
        }
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
          const float* src = comb + (w * 8 + r) * C::CSTRIDE + d0;
#pragma unroll
          for (int i = 0; i < PER; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(src + i);
            acc[i] += wgt[w] * x.x;
            acc[i + 1] += wgt[w] * x.y;
            acc[i + 2] += wgt[w] * x.z;
            acc[i + 3] += wgt[w] * x.w;
          }
        }
        const int hq = h * G + 8 * half + r;
        if (whole) {
          const float inv = den > 0.f ? vsc / den : (den == den ? 0.f : den);  // a NaN stays one
          uint16_t* out = p.out + (static_cast<int64_t>(sw.b) * p.heads + hq) * DV + d0;
          uint32_t pk[PER / 2];
#pragma unroll
          for (int i = 0; i < PER / 2; ++i) pk[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
          if (PER == 8)
            *reinterpret_cast<uint4*>(out) = make_uint4(pk[0], pk[1], pk[2 % (PER / 2)], pk[3 % (PER / 2)]);
          else
            *reinterpret_cast<uint2*>(out) = make_uint2(pk[0], pk[1]);
          if (p.lse && d0 == 0)
            p.lse[static_cast<int64_t>(hq) * p.batch + sw.b] =
                den > 0.f ? top * kLn2p + logf(den) : (den == den ? -INFINITY : den);
        } else {
          const int64_t at = static_cast<int64_t>(part) * p.heads + hq;
#pragma unroll
          for (int i = 0; i < PER; i += 4)
            *reinterpret_cast<float4*>(ws.o + at * DV + d0 + i) =
                make_float4(acc[i] * vsc, acc[i + 1] * vsc, acc[i + 2] * vsc, acc[i + 3] * vsc);
          if (d0 == 0) ws.ml[at] = make_float2(top, den);
        }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    left -= np;
    page = 0;
    sw = nx;
  }
}

// Adds up the parts of one sequence that crosses columns, for one query head:
// CTA (column, head); warp w takes parts w, w + 4, ...
template <int DV>
__global__ void __launch_bounds__(128) decode_join_kernel(const __grid_constant__ PagedDecodeParams p,
                                                          const Workspace ws) {
  constexpr int PER = DV / 32;
  __shared__ float so[4][DV];
  __shared__ float2 sml[4];
  grid_wait();
  const int c = blockIdx.x, hq = blockIdx.y;
  const JoinDesc d = ws.desc[c];
  if (d.b < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto at = [&](int i) {
    return static_cast<int64_t>(i == 0 ? (c - 1) * 2 + d.slot : (c - 1 + i) * 2) * p.heads + hq;
  };
  float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) acc[j] = 0.f;
#pragma unroll 4
  for (int i = warp; i < d.n; i += 4) {
    const float2 x = ws.ml[at(i)];
    float v[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = ws.o[at(i) * DV + lane + 32 * j];
    const float top = fmaxf(m, x.x);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - top), w = x.x == -INFINITY ? 0.f : ex2_approx(x.x - top);
    l = l * f + x.y * w;
#pragma unroll
    for (int j = 0; j < PER; ++j) acc[j] = acc[j] * f + v[j] * w;
    m = top;
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) so[warp][lane + 32 * j] = acc[j];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x >= DV) return;
  float top = -INFINITY, den = 0.f, x = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, sml[w].x);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = sml[w].x == -INFINITY ? 0.f : ex2_approx(sml[w].x - top);
    den += f * sml[w].y;
    x += f * so[w][threadIdx.x];
  }
  const float inv = den > 0.f ? 1.f / den : (den == den ? 0.f : den);
  p.out[(static_cast<int64_t>(d.b) * p.heads + hq) * DV + threadIdx.x] =
      static_cast<uint16_t>(pack_bf16x2(x * inv, 0.f) & 0xFFFFu);
  if (p.lse && threadIdx.x == 0)
    p.lse[static_cast<int64_t>(hq) * p.batch + d.b] = den > 0.f ? top * kLn2p + logf(den) : (den == den ? -INFINITY : den);
}

// Columns of the work split: cols x kv_heads CTAs in whole waves of the CTAs
// that are resident at once.  The smallest number of waves that leaves at most 4%
// of the places empty (8 kv heads: one wave of 38 columns; 128: three
// waves of 7), or the fullest of up to four.
int decode_cols(int kv_heads, int places) {
  int best = 1;
  double best_fill = 0.0;
  for (int w = 1; w <= 4; ++w) {
    const int c = w * places / kv_heads;
    if (c < 1) continue;
    const double fill = static_cast<double>(c) * kv_heads / (w * places);
    if (fill > best_fill + 1e-9) {
      best_fill = fill;
      best = c;
    }
    if (best_fill >= 0.96) break;
  }
  return best;
}

template <int DQ, int DV, bool F8, int NG>
cudaError_t launch_t(const PagedDecodeParams& p, const CUtensorMap* maps, const Workspace& ws, int cols,
                     cudaStream_t stream) {
  using C = Cfg<DQ, DV, F8, NG>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    e = cudaFuncSetAttribute(paged_decode_kernel<DQ, DV, F8, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  e = launch_overlapped(paged_decode_kernel<DQ, DV, F8, NG>, dim3(cols * p.kv_heads), kThreads, C::SMEM, stream, maps[0],
                        maps[1], maps[2], maps[3], p, ws, cols);
  if (e != cudaSuccess || cols == 1) return e;
  return launch_overlapped(decode_join_kernel<DV>, dim3(cols, p.heads), 128, 0, stream, p, ws);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t paged_decode_ws_bytes(int32_t, int heads, int kv_heads, int dq, int dv, int num_sms) {
  const int ng = heads / kv_heads > 8 ? 2 : 1;  // the larger of the two cache types' needs
  const size_t cols = std::max(decode_cols(kv_heads, num_sms * ctas_per_sm(dq, dv, false, ng)),
                               decode_cols(kv_heads, num_sms * ctas_per_sm(dq, dv, true, ng)));
  if (cols == 1) return 0;
  return align256(cols * 2 * heads * dv * 4) + align256(cols * 2 * heads * 8) + align256(cols * sizeof(JoinDesc));
}

cudaError_t launch_paged_decode(const PagedDecodeParams& p, bool fp8, const CUtensorMap* maps, void* workspace,
                                int num_sms, cudaStream_t stream) {
  const int cols =
      decode_cols(p.kv_heads, num_sms * ctas_per_sm(p.dq, p.dv, fp8, p.heads / p.kv_heads > 8 ? 2 : 1));
  Workspace ws = {};
  if (cols > 1) {
    uint8_t* at = static_cast<uint8_t*>(workspace);
    ws.o = reinterpret_cast<float*>(at);
    at += align256(static_cast<size_t>(cols) * 2 * p.heads * p.dv * 4);
    ws.ml = reinterpret_cast<float2*>(at);
    at += align256(static_cast<size_t>(cols) * 2 * p.heads * 8);
    ws.desc = reinterpret_cast<JoinDesc*>(at);
  }
#define VPP_CASE(DQ, DV)                                                             \
  if (p.dq == DQ && p.dv == DV)                                                      \
    return p.heads / p.kv_heads > 8                                                  \
               ? (fp8 ? launch_t<DQ, DV, true, 2>(p, maps, ws, cols, stream)         \
                      : launch_t<DQ, DV, false, 2>(p, maps, ws, cols, stream))       \
               : (fp8 ? launch_t<DQ, DV, true, 1>(p, maps, ws, cols, stream)         \
                      : launch_t<DQ, DV, false, 1>(p, maps, ws, cols, stream));
  VPP_CASE(64, 64)
  VPP_CASE(64, 128)
  VPP_CASE(128, 64)
  VPP_CASE(128, 128)
  VPP_CASE(192, 64)
  VPP_CASE(192, 128)
#undef VPP_CASE
  return cudaErrorInvalidValue;
}

}  // namespace vpp
