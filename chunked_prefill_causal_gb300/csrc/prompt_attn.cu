// prompt_attn.cu -- causal attention of whole prompts, packed one after the
// other, straight from the projection's q, k and v (no cache).
//
// "VPP: Virtual Pipeline Parallelism for Efficient Chunked Prefill in
// Long-Context LLM Inference" (technical review), §2.2, Eq. (1): token i of a
// sequence attends to that sequence's tokens <= i.
//
// The inner loop is that of the chunk-attention kernel (chunk_attn_impl.cuh): two
// 128-row query tiles per CTA take turns on the tensor core, each row of a tile
// is one softmax thread, P is read from TMEM by the P V product.  Around it:
//
// Items.  An item is one or two query tiles (T = floor(128 / G) tokens of the G heads of
// one kv head each) of one sequence, and the grid has a CTA for each.  The
// sequences are read from cu_seqlens on the device; they are ordered by length
// class, longest first, and a sequence's items from its last tokens to its first,
// head by head: the heaviest start first, and the items that read the same keys
// and values run at the same time.  (Ordered by their weight alone, equal prompts
// read each key from HBM once per tile of queries: 32768 tokens in prompts of
// 512 moved 1.25 GB for the 0.4 GB that there are.)  Where the keys and values of a
// sequence's heads together take more than half of L2, all its items of 32 heads come
// before the next 32 heads': with 128 heads of their own keys and 192 dims, two prompts
// of 4096 tokens take 1068 us, all heads together 1172; four of 2048 604 and 654; three
// of 720 to 1026 146 and 154.
//
// Persistent CTAs.  A resident CTA takes over another one of the grid that has not
// started (cluster launch control), so the items go to whichever SM is free, in
// about their order, without a counter in memory.  The chunk kernel's one-item CTAs cost
// about 8 us each besides their keys (launch, TMEM, first loads, drain, output),
// most of the time of short prompts; here the next item's Q and K/V copies and its
// first Q K^T run while the last softmax and the output of the current one do.
//
//   warp 0      TMA producer (Q of the item, then K and V tiles, ring of 16 KB slots)
//   warp 1, 3   MMA issuers of query tiles A and B, taking turns
//   warp 2      TMEM; finds the next item while one is under way and hands it out
//               through shared memory; zeroes the V rows of other
//               sequences in an item's last tile (P = 0 times whatever they hold
//               must stay 0; their K rows are masked before the softmax)
//   warps 4-7, 8-11   softmax and output of tiles A and B
//
// The two tiles of a pair may need different numbers of key tiles (nA <= nB; B is
// absent when the sequence ends in A), and each runs its own number.
//
// Rounding: a row's P is rounded to bf16 as the P V operand (relative 2^-8, against V
// in bf16); its sum, the denominator, keeps the float32 values, as O and the scores do.
//
// Bound by the tensor core and the softmax that feeds it for long prompts: one of
// 16384 tokens, 32/8 heads of 128, takes 1350 to 1380 us on a GB300, 1593 to 1629
// TFLOP/s (83 to 85% of the cuBLAS rate; tensor pipe active 68% of the cycles, issue
// slots 42%).  Bound by the chain of one item (first loads, first softmax, drain,
// output: 2.5 us beside its keys) for short ones: 24 prompts of 5 to 2500 tokens take
// 106 us (984 TFLOP/s, tensor pipe 47%).  At 192 dims the ring holds a K tile, its V
// tile and the next K tile, no more, and each item starts by loading 96 KB of Q: three
// prompts of 720 to 1026 tokens, 128 heads of their own keys, take 146 us, 2.2 times
// their bytes' time.
#include <algorithm>
#include <climits>

#include "chunk_attn_impl.cuh"
#include "prompt_attn.cuh"

namespace vpp {
namespace {

using namespace attn_detail;

constexpr int kEntries = 4;  // items handed out at most (two ahead)
constexpr int kAskTiles = 6;  // key tiles left of an item when the next one is asked for

// Kv heads of a sequence that go together where all of them would take more than half
// of L2 (129 MB, which queries and output pass through as well).
constexpr int kHeadGroup = 32;
constexpr int64_t kKeptBytes = 64ll << 20;

struct Item {
  int start, len;  // the sequence's rows
  int tok0;        // first token of tile A
  int g;           // kv head
  int na, nb;      // key tiles of A and of B (nb = 0: no B)
  int pad[2];
};

// PAIR: two query tiles a CTA, one CTA per SM.  Otherwise one tile, two CTAs.
template <int DQ, int DV, bool PAIR>
struct PShape {
  using S = Shape<DQ, DV, false>;
  static constexpr int TILES = PAIR ? 2 : 1;
  static constexpr int CTAS = PAIR ? 1 : 2;  // per SM
  static constexpr int NQC = S::NQC, NVC = S::NVC;
  static constexpr int QBYTES = TILES * NQC * kSubTileBytes;
  static constexpr int SOFTMAX = 128 * TILES;
  static constexpr int THREADS = 128 + SOFTMAX;
  // 228 KB per SM, 1 KB of it per CTA for the system; 768 bytes for the
  // entries and barriers.
  static constexpr int LIMIT = 228 * 1024 / CTAS - 1024;
  static constexpr int FIT = (LIMIT - QBYTES - 768) / kSubTileBytes;
  static constexpr int NSLOT = FIT > 12 ? 12 : FIT;
  static constexpr int NB = NSLOT;
  static_assert(NSLOT >= NQC + NVC, "ring must hold one K and one V tile");
  static constexpr int REGS_LOW = PAIR ? kRegsLow : 80;
  static constexpr int REGS_HIGH = PAIR ? kRegsHigh : 176;
  static_assert(128 * REGS_LOW + SOFTMAX * REGS_HIGH <= THREADS * (PAIR ? 168 : 128), "register split exceeds the launch");
  static constexpr int TMEM_COLS = 256 * TILES;  // S tiles, then O tiles
  static constexpr int PV0 = S::PV0, KP0 = S::KP0;
  static constexpr bool SPLIT_P = S::SPLIT_P, EARLY_V = S::EARLY_V;
  static constexpr int B_Q = 0, B_QE = 1, B_S = 2, B_P = 4, B_P1 = 6, B_O = 8, B_FINAL = 10, B_END = 12, B_IF = 13,
                       B_IE = B_IF + kEntries, B_FULL = B_IE + kEntries, B_EMPTY = B_FULL + NB, B_TMP = B_EMPTY + NB,
                       B_CLC = B_TMP + NB, NBARS = B_CLC + 1;
  static constexpr int SMEM = QBYTES + NSLOT * kSubTileBytes + (kEntries + 1) * 32 + NBARS * 8 + 16 + 32 * 4;
  static_assert(SMEM <= LIMIT && SMEM <= kSmemLimit, "shared memory budget");
  // Tile t of the load order (K_0, V_0, K_1, ...): first ring position and slots.
  __device__ __forceinline__ static int tile_pos(int t) { return S::tile_pos(t); }
  __device__ __forceinline__ static int tile_slots(int t) { return S::tile_slots(t); }
};

// x / d, with d's multiplier and shift from the host (see divide_by()).
__device__ __forceinline__ int quotient(uint32_t x, uint64_t mul, int shift) {
  return static_cast<int>((x * mul) >> shift);
}

// Items of a sequence of rows [s, e): 0 where the range is not one of the call's rows.
__device__ __forceinline__ int items_of(const PromptParams& p, int s, int e) {
  return s < 0 || e < s || e > p.total ? 0 : quotient(e - s + p.item_tokens - 1, p.item_mul, p.item_shift);
}

// Length class of a sequence of n > 0 items: from the longest (0) on, powers of two.
__device__ __forceinline__ int class_of(int n) { return __clz(n); }

// Adds up the items of each class, by all threads of the CTA.  (Compact code: it runs
// once, and what it takes is fetching it.)
__device__ __forceinline__ void count_classes(const PromptParams& p, int* sums) {
#pragma unroll 1
  for (int64_t b = threadIdx.x; b < p.batch; b += blockDim.x) {
    const int s = __ldg(p.cu + b), e = __ldg(p.cu + b + 1);
    const int n = items_of(p, s, e);
    if (n > 0)
      atomicAdd(&sums[class_of(n)], n);
    else if (s != e || s < 0 || e > p.total)  // (by every CTA: which ones start is the hardware's choice)
      record_status(p.status, kStatusInvalid);
  }
}

// The work list, by one warp: the classes from the longest on, the sequences of a
// class in their order.  A lane holds four of 128 sequences; items mostly come in
// increasing order, so most are found among those at hand, and an earlier one starts
// the scan over.  (With 32 at hand, and the classes found by two scans of one warp,
// 1024 prompts of 32 tokens took 157 us, now 126; 256 of 128 with 8/8 heads 50, now 45.)
struct Finder {
  const PromptParams& p;
  int lane;
  int upto;          // items of the classes up to this lane's
  int cls, before;   // the class at hand, items of the ones before it
  int base, scan;    // first sequence at hand, and the class's items before it
  int row[5], n[4];  // this lane's sequences: first rows (and that behind), items in the class
  int mine, inc;     // their sum, and with those of the lanes before
  __device__ __forceinline__ Finder(const PromptParams& p_, const int* sums)
      : p(p_), lane(threadIdx.x & 31), cls(-1), before(0), base(0), scan(0) {
    upto = scan_lanes(sums[lane]);
  }
  __device__ __forceinline__ int scan_lanes(int x) const {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int j = 0; j < 5; ++j)
      row[j] = __ldg(p.cu + min(static_cast<int64_t>(base) + 4 * lane + j, static_cast<int64_t>(p.batch)));
    mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = items_of(p, row[j], row[j + 1]);
      n[j] = m > 0 && class_of(m) == cls ? m : 0;
      mine += n[j];
    }
    inc = scan_lanes(mine);
  }
  // Item i: its sequence's rows and its index in the sequence (the last tokens
  // come first); false when there is no such item.
  __device__ __forceinline__ bool find(int i, int* first, int* length, int* index) {
    const uint32_t in = __ballot_sync(0xffffffffu, i < upto);
    if (!in) return false;
    const int l = __ffs(in) - 1;
    const int longer = l > 0 ? __shfl_sync(0xffffffffu, upto, l - 1) : 0;
    if (cls != l || i < longer + scan) {
      cls = l;
      before = longer;
      base = scan = 0;
      load();
    }
    const int want = i - before;
    while (true) {
      const uint32_t hit = __ballot_sync(0xffffffffu, want < scan + inc);
      if (hit) {
        const int from = __ffs(hit) - 1;
        int at = want - (scan + inc - mine), s = row[0], e = row[1], m = n[0];
#pragma unroll
        for (int j = 1; j < 4; ++j)
          if (at >= m) {
            at -= m;
            s = row[j];
            e = row[j + 1];
            m = n[j];
          }
        *first = __shfl_sync(0xffffffffu, s, from);
        *length = __shfl_sync(0xffffffffu, at >= 0 && at < m ? e - s : 0, from);
        *index = __shfl_sync(0xffffffffu, m - 1 - at, from);
        return *length > 0;  // (always, unless the ranges overlap so that the counts overflow)
      }
      scan += __shfl_sync(0xffffffffu, inc, 31);
      base += 128;
      if (base >= p.batch) return false;  // (likewise)
      load();
    }
  }
};

// Asks the hardware for the next CTA of this grid that has not started, to be
// run here in its place; the answer (16 bytes) arrives on the mbarrier.
__device__ __forceinline__ void clc_request(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   answer),
               "r"(bar)
               : "memory");
}

// Index of the CTA that was given, -1 when all have started.
__device__ __forceinline__ int clc_answer(uint32_t answer) {
  int x;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 a, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "mov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, a;\n\t}"
      : "=r"(x)
      : "r"(answer)
      : "memory");
  return x;
}

// w[i] of lane a (of each group of four) becomes w[a] of lane i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4][4], int a) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit *= 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, (a & bit) ? w[i][c] : w[i | bit][c], bit);
        if (a & bit) w[i][c] = got; else w[i | bit][c] = got;
      }
    }
  }
}

// Scores of 32 keys of this thread's row; those past `lim` leave the softmax.
__device__ __forceinline__ void load_scores(uint32_t taddr, int key, int lim, float (&s)[32]) {
  uint32_t u[32];
  tmem_ld32(taddr, u);
  tmem_ld_wait();
#pragma unroll
  for (int k = 0; k < 32; ++k) s[k] = __uint_as_float(u[k]);
  if (__any_sync(0xffffffffu, key + 31 > lim)) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (key + k > lim) s[k] = -INFINITY;
  }
}

template <int DQ, int DV, bool PAIR>
__global__ void __launch_bounds__(PShape<DQ, DV, PAIR>::THREADS, PShape<DQ, DV, PAIR>::CTAS)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PromptParams p) {
  using S = PShape<DQ, DV, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + S::QBYTES;
  Item* entries = reinterpret_cast<Item*>(sRing + S::NSLOT * kSubTileBytes);
  uint8_t* clc = reinterpret_cast<uint8_t*>(entries + kEntries);  // 16 bytes
  uint64_t* bars = reinterpret_cast<uint64_t*>(clc + 32);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + S::NBARS);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
  volatile int* turn = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* sums = reinterpret_cast<int*>(tmem_slot + 4);  // items of the 32 length classes
  auto bar = [&](int i) { return smem_u32(&bars[i]); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.heads / p.kv_heads;
  const int T = kTileM / G;  // tokens per query tile

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    *turn = 0;
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (threadIdx.x < S::NBARS) {
    const int i = threadIdx.x;
    int count = 1;
    if (i == S::B_QE) count = S::TILES;
    if (i >= S::B_P && i < S::B_O) count = 128;
    if (i == S::B_END) count = 5 * S::TILES;                            // the softmax warps and the MMA issuers
    if (i >= S::B_IE && i < S::B_FULL) count = 1 + 5 * S::TILES;        // producer, issuers, softmax warps
    if (i >= S::B_EMPTY && i < S::B_TMP) count = S::TILES;              // released by the MMA issuers
    mbar_init(bar(i), count);
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), S::TMEM_COLS);
    tmem_relinquish();
  }
  if (threadIdx.x >= 32 && threadIdx.x < 64) sums[lane] = 0;
  grid_wait();
  __syncthreads();
  count_classes(p, sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  // Item i of this CTA, as one thread (producer, issuer) reads it.
  auto read_item = [&](int i, Item* it) {
    if (!mbar_wait(bar(S::B_IF + i % kEntries), (i / kEntries) & 1, p.status, abort_flag)) return false;
    *it = entries[i % kEntries];
    return it->len > 0;
  };
  auto take = [&](int i, Item* it) {
    if (!read_item(i, it)) return false;
    mbar_arrive(bar(S::B_IE + i % kEntries));
    return true;
  };

  if (warp < 4) {
    regs_dec<S::REGS_LOW>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA producer
      bool ok = true;
      int base = 0;    // tile pairs (K and V) of the items before
      int issued = 0;  // tiles whose loads were started
      int rq = 0;      // next tile whose release has not been observed
      uint32_t tmp_phase = 0u, tmp_last = 0u;  // parity of B_TMP's next use; tiles that landed there last
      int n_items = 0;
      Item it;
      for (int i = 0; ok && read_item(i, &it); ++i) {
        const int n = max(it.na, it.nb);
        if (i > 0 && !(ok = mbar_wait(bar(S::B_QE), (i - 1) & 1, p.status, abort_flag))) break;
        const int tiles_q = it.nb > 0 ? 2 : 1;
        // (a group that does not divide 128 leaves the last rows of a tile unused)
        mbar_arrive_expect_tx(bar(S::B_Q), tiles_q * S::NQC * G * T * 128);
        for (int x = 0; x < tiles_q; ++x)
          for (int c = 0; c < S::NQC; ++c)
            tma_load_4d(smem_u32(sQ + (x * S::NQC + c) * kSubTileBytes), &tm_q, bar(S::B_Q), c * 64, 0, it.g,
                        it.start + it.tok0 + x * T);
        n_items = i + 1;
        for (int j = 0; ok && j < n; ++j) {
          // (the next item is asked for when six tiles are left)
          if (j == max(0, n - kAskTiles)) mbar_arrive(bar(S::B_IE + i % kEntries));
          for (int part = 0; part < 2; ++part) {  // K, then V
            const int t = 2 * (base + j) + part;
            const int pos = S::tile_pos(t);
            const int nsub = S::tile_slots(t);
            // Tiles are released in load order: wait until every tile that used
            // these slots, and the tile that last used this barrier, is released.
            while (rq < t && (rq <= t - S::NB || S::tile_pos(rq) < pos + nsub - S::NSLOT)) {
              if (!(ok = mbar_wait(bar(S::B_EMPTY + rq % S::NB), (rq / S::NB) & 1u, p.status, abort_flag))) break;
              ++rq;
            }
            if (!ok) break;
            // V rows past the sequence: the tile lands on B_TMP and warp 2
            // completes it.
            const bool fix = part == 1 && j == n - 1 && it.len - j * kTileN < kTileN;
            const uint32_t fb = bar((fix ? S::B_TMP : S::B_FULL) + t % S::NB);
            if (fix) {
              tmp_phase ^= 1u << (t % S::NB);
              tmp_last |= 1u << (t % S::NB);
            } else {
              tmp_last &= ~(1u << (t % S::NB));
            }
            const CUtensorMap* m = part == 0 ? &tm_k : &tm_v;
            mbar_arrive_expect_tx(fb, nsub * kSubTileBytes);
            for (int c = 0; c < nsub; ++c) {
              const uint32_t d = smem_u32(sRing + ((pos + c) % S::NSLOT) * kSubTileBytes);
              tma_load_3d(d, m, fb, c * 64, it.g, it.start + j * kTileN);
              tma_load_3d(d + kSubTileBytes / 2, m, fb, c * 64, it.g, it.start + j * kTileN + kBlockTokens);
            }
            issued = t + 1;
          }
        }
        base += n;
      }
      if (*abort_flag) {
        // Let every copy this thread started land before the CTA exits.
        for (int t = issued > S::NB ? issued - S::NB : 0; t < issued; ++t) {
          const int b = t % S::NB;
          if (tmp_last & (1u << b))
            mbar_wait_for(bar(S::B_TMP + b), ((tmp_phase >> b) & 1u) ^ 1u, kCleanupNs);
          else
            mbar_wait_for(bar(S::B_FULL + b), (t / S::NB) & 1u, kCleanupNs);
        }
        if (n_items > 0) mbar_wait_for(bar(S::B_Q), (n_items - 1) & 1, kCleanupNs);
      }
    } else if (warp == 2) {
      // --------------------------------------- items, and V rows of other sequences
      Finder finder(p, sums);
      int requests = 0;
      bool ok = true;
      Item it;
      // Item of CTA `idx`; false if it has none (the grid's size is an upper bound).
      auto item_of = [&](int idx) {
        const int item = quotient(idx, p.head_mul, p.head_shift);
        int index;
        if (!finder.find(item, &it.start, &it.len, &index)) return false;
        it.g = idx - item * p.kv_heads;
        if (p.kv_heads > kHeadGroup && static_cast<int64_t>(it.len) * p.kv_heads * (DQ + DV) * 2 > kKeptBytes) {
          // groups of heads, the sequence's items of one group before the next one's
          const int n = (it.len + S::TILES * T - 1) / (S::TILES * T);
          const int at = (n - 1 - index) * p.kv_heads + it.g;  // in the sequence's order
          const int first = at / (n * kHeadGroup) * kHeadGroup;
          const int heads = min(kHeadGroup, p.kv_heads - first);
          const int rest = at - first * n;
          index = n - 1 - rest / heads;
          it.g = first + rest % heads;
        }
        it.tok0 = index * S::TILES * T;
        it.na = (min(it.tok0 + T, it.len) + kTileN - 1) / kTileN;
        it.nb = PAIR && it.tok0 + T < it.len ? (min(it.tok0 + 2 * T, it.len) + kTileN - 1) / kTileN : 0;
        return true;
      };
      // The next item: of a CTA of the grid that has not started, until one has an
      // item or none is left.  (The order in which they are given is the
      // hardware's; it is nearly, not always, that of their indexes.)
      auto next_item = [&]() {
        while (ok) {
          __syncwarp();
          if (lane == 0) {
            fence_proxy_async_smem();  // after the reads of the answer before
            mbar_arrive_expect_tx(bar(S::B_CLC), 16);
            clc_request(smem_u32(clc), bar(S::B_CLC));
          }
          ok = warp_wait(bar(S::B_CLC), requests & 1, p.status, abort_flag);
          if (!ok) mbar_wait_for(bar(S::B_CLC), requests & 1, kCleanupNs);  // lands before the CTA exits
          ++requests;
          const int idx = ok ? clc_answer(smem_u32(clc)) : -1;
          if (idx < 0) break;
          if (item_of(idx)) return;
        }
        it.len = 0;
      };
      int published = 0;
      auto publish = [&]() {
        if (lane == 0) {
          entries[published % kEntries] = it;
          mbar_arrive(bar(S::B_IF + published % kEntries));
        }
        __syncwarp();
        ++published;
      };
      if (!item_of(blockIdx.x)) next_item();
      publish();
      int base = 0;
      uint32_t tmp_phase = 0u;
      for (int i = 0; ok; ++i) {
        const Item cur = entries[i % kEntries];
        if (cur.len == 0) break;
        const int n = max(cur.na, cur.nb);
        // V rows past the sequence in the item's last tile
        auto zero_rows = [&]() {
          const int t = 2 * (base + n) - 1, tb = t % S::NB, pos = S::tile_pos(t);
          const int r0 = cur.len - (n - 1) * kTileN;
          if (r0 >= kTileN) return;
          ok = warp_wait(bar(S::B_TMP + tb), (tmp_phase >> tb) & 1u, p.status, abort_flag);
          if (!ok) return;
          tmp_phase ^= 1u << tb;
          for (int u = r0 * 8 + lane; u < kTileN * 8; u += 32)  // 16-byte units of rows r0 .. 127
#pragma unroll
            for (int c = 0; c < S::NVC; ++c)
              *reinterpret_cast<uint4*>(sRing + ((pos + c) % S::NSLOT) * kSubTileBytes + u * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(S::B_FULL + tb));
        };
        // Further items are asked for once every role has begun this one and its
        // copies are near its end: the next one, or two when this is short (an
        // answer, its sequence and its first copies take as long as a short item:
        // 1024 prompts of 32 tokens take 156 us with one ahead, 126 us with two).  A CTA
        // that asks earlier holds items that others could have run: one prompt of 2000
        // tokens takes 41.2 us asking at an item's start, 32.4 us with six tiles left, four
        // of 2048 with 128 heads of 192 dims 616 and 604 us; with one tile left the
        // latter take 640 us.
        // A short item's own rows come first.
        const bool is_short = n <= 2;
        if (is_short) zero_rows();
        if (ok) ok = warp_wait(bar(S::B_IE + i % kEntries), (i / kEntries) & 1, p.status, abort_flag);
        while (ok && it.len > 0 && published <= i + (is_short ? 2 : 1)) {
          next_item();
          if (ok) publish();
        }
        if (ok && !is_short) zero_rows();
        base += n;
      }
    } else if ((warp == 1 || (PAIR && warp == 3)) && lane == 0) {
      // ---------------------------------------------------- MMA issuer
      const int x = warp == 1 ? 0 : 1;
      const uint64_t dq0 = sdesc_sw128(smem_u32(sQ + x * S::NQC * kSubTileBytes), 16, 1024);
      const uint64_t dk0 = sdesc_sw128(smem_u32(sRing), 16, 1024);             // K-major
      const uint64_t dv0 = sdesc_sw128(smem_u32(sRing), kSubTileBytes, 1024);  // MN-major
      constexpr uint32_t kSub16 = kSubTileBytes >> 4;
      const uint32_t tS = tbase + x * kTileN;
      const uint32_t tO = tbase + S::TILES * kTileN + x * DV;
      bool ok = true;
      int base = 0;    // tile pairs of the items before
      int mine = 0;    // S tiles of this query tile before
      int number = 0;  // blocks of both issuers before
      int kslot0 = 0;  // ring slot of the item's first K tile
      Item it;
      for (int i = 0; ok && take(i, &it); ++i) {
        const int n = max(it.na, it.nb);
        const int nx = x == 0 ? it.na : it.nb, ny = x == 0 ? it.nb : it.na;
        const int ba = it.na + 1, bb = it.nb > 0 ? it.nb + 1 : 0;  // blocks of A and of B
        if (nx > 0) {
          if (!(ok = mbar_wait(bar(S::B_Q), i & 1, p.status, abort_flag))) break;
          int kslot = kslot0;
          int vslot = kslot0 + S::NQC - (S::NQC + S::NVC);  // becomes V_0's slot at j = 1
          if (vslot < 0) vslot += S::NSLOT;
          // Block j = [PV(x, j-1) if j > 0][QK(x, j) if j < nx].  The blocks run in the
          // order A0 B0 A1 B1 ..., A's last, the rest of B's.
          for (int j = 0; ok && j <= nx; ++j) {
            const int tk = 2 * (base + j);  // tile index of K_j
            const int tv = tk - 1;          // tile index of V_{j-1}
            const int my_turn = number + (x == 0 ? j + min(j, bb) : j + min(j + 1, ba));
            if (j > 0) {
              kslot += S::NQC + S::NVC;
              if (kslot >= S::NSLOT) kslot -= S::NSLOT;
              vslot += S::NQC + S::NVC;
              if (vslot >= S::NSLOT) vslot -= S::NSLOT;
              if (!(ok = mbar_wait(bar(S::B_FULL + tv % S::NB), (tv / S::NB) & 1u, p.status, abort_flag))) break;
              if (!(ok = mbar_wait(bar(S::B_P + x), (mine + j - 1) & 1, p.status, abort_flag))) break;
              tc_fence_after();
            }
            if (j < nx &&
                !(ok = mbar_wait(bar(S::B_FULL + tk % S::NB), (tk / S::NB) & 1u, p.status, abort_flag)))
              break;
            // Take the partner's turn: a tight spin on the shared counter (the abort flag
            // and the time limit are checked every 256 polls).
            if (PAIR && *turn != my_turn) {
              const uint64_t t0 = globaltimer_ns();
              for (uint32_t k = 1; *turn != my_turn; ++k) {
                if ((k & 255u) != 0) continue;
                if (*abort_flag) { ok = false; break; }
                if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
                  record_status(p.status, kStatusTimeout);
                  *abort_flag = 1u;
                  ok = false;
                  break;
                }
              }
              if (!ok) break;
            }
            if (j > 0) {
              // (V tiles of two slots never wrap when everything comes in twos)
              constexpr bool kTwos = S::NQC % 2 == 0 && S::NVC == 2 && S::NSLOT % 2 == 0;
              const bool adjacent = S::NVC == 1 || kTwos || vslot + S::NVC <= S::NSLOT;
              auto pv_steps = [&](int k0, int k1) {
                if (adjacent) {
                  const uint64_t vb = dv0 + vslot * kSub16;
#pragma unroll
                  for (int k = k0; k < k1; ++k)
                    umma_ts(tO, tS + 8 * k, vb + k * (2048 >> 4), S::S::IDESC_PV, (j > 1 || k > 0) ? 1u : 0u);
                } else {
#pragma unroll
                  for (int k = k0; k < k1; ++k)
#pragma unroll
                    for (int h = 0; h < S::NVC; ++h) {
                      const int vs = vslot + h < S::NSLOT ? vslot + h : vslot + h - S::NSLOT;
                      umma_ts(tO + 64 * h, tS + 8 * k, dv0 + vs * kSub16 + k * (2048 >> 4), S::S::IDESC_PV64,
                              (j > 1 || k > 0) ? 1u : 0u);
                    }
                }
              };
              pv_steps(0, S::PV0);
              if (S::SPLIT_P) {
                if (!(ok = mbar_wait(bar(S::B_P1 + x), (mine + j - 1) & 1, p.status, abort_flag))) break;
                tc_fence_after();
                pv_steps(S::PV0, kTileN / 16);
              }
              if (S::EARLY_V) umma_commit(bar(S::B_EMPTY + tv % S::NB));
            }
            if (j < nx) {
              // The turn goes to the partner before the last four MMAs: its
              // first ones then queue behind them.
#pragma unroll
              for (int c = 0; c < S::NQC; ++c) {
                const int ks = kslot + c < S::NSLOT ? kslot + c : kslot + c - S::NSLOT;
                const uint64_t kb = dk0 + ks * kSub16;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (PAIR && c == S::NQC - 1 && k == 0) *turn = my_turn + 1;
                  umma_ss(tS, dq0 + c * kSub16 + 2 * k, kb + 2 * k, S::S::IDESC_QK, (c | k) ? 1u : 0u);
                }
              }
              umma_commit(bar(S::B_S + x));
              umma_commit(bar(S::B_EMPTY + tk % S::NB));
              if (PAIR && j >= ny) mbar_arrive(bar(S::B_EMPTY + tk % S::NB));  // the partner does not read this tile
              if (j == nx - 1) {
                umma_commit(bar(S::B_QE));
                if (PAIR && ny == 0) mbar_arrive(bar(S::B_QE));
              }
            } else if (PAIR) {
              *turn = my_turn + 1;
            }
            if (j > 0) {
              if (!S::EARLY_V) umma_commit(bar(S::B_EMPTY + tv % S::NB));
              if (PAIR && j - 1 >= ny) mbar_arrive(bar(S::B_EMPTY + tv % S::NB));
            }
            if (j == nx) umma_commit(bar(S::B_O + x));
          }
        }
        base += n;
        mine += nx;
        number += ba + bb;
        kslot0 = (kslot0 + n * (S::NQC + S::NVC)) % S::NSLOT;
      }
      if (*abort_flag) {
        // Every MMA issued so far must finish before TMEM is freed.
        umma_commit(bar(S::B_FINAL + x));
        mbar_wait_for(bar(S::B_FINAL + x), 0, kCleanupNs);
      }
    }
  } else {
    regs_inc<S::REGS_HIGH>();
    // ------------------------------------------------------ softmax + output
    const int x = (warp - 4) >> 2;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const int row_tok = row / G, row_head = row % G;
    const uint32_t lane_base = tbase + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t tS = lane_base + x * kTileN;
    const uint32_t tO = lane_base + S::TILES * kTileN + x * DV;
    const float sl = p.scale_log2;
    bool ok = true;
    int mine = 0;     // S tiles of this query tile before
    int outputs = 0;  // items with this query tile before
    for (int i = 0; ok; ++i) {
      if (!(ok = warp_wait(bar(S::B_IF + i % kEntries), (i / kEntries) & 1, p.status, abort_flag))) break;
      const Item it = entries[i % kEntries];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::B_IE + i % kEntries));
      if (it.len == 0) break;
      const int n = x == 0 ? it.na : it.nb;
      if (n == 0) continue;
      const int tok = it.tok0 + x * T + row_tok;
      const int lim = min(tok, it.len - 1);  // last visible key (inclusive)
      const int warp_lim0 = __shfl_sync(0xffffffffu, lim, 0), warp_lim = __shfl_sync(0xffffffffu, lim, 31);
      float m = -INFINITY;  // running max of score * scale * log2(e)
      float l = 0.f;        // running denominator, relative to 2^m
      for (int j = 0; j < n; ++j) {
        // Takes the tile's row maximum into the reference m, which moves only when
        // it has grown by more than 2^8 (exact either way: numerator and
        // denominator share it); O and the denominator are then rescaled.  O is
        // idle here: PV(x, j-1) completed before S(x, j) was committed, and
        // PV(x, j) waits for this group's P.  True if a row of the warp moved.
        auto raise = [&](float mx) {
          const float m_new = fmaxf(m, mx * sl);
          const bool need = m_new > m + kRescaleThreshold || (m == -INFINITY && m_new > -INFINITY);
          if (!__any_sync(0xffffffffu, need)) return false;
          const float f = need ? ex2_approx(m - m_new) : 1.f;
          if (need) {
            l *= f;
            m = m_new;
          }
          if (j == 0) return true;
#pragma unroll 1
          for (int q = 0; q < DV / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st32(tO + 32 * q, o);
          }
          return true;
        };
        if (!(ok = warp_wait(bar(S::B_S + x), (mine + j) & 1, p.status, abort_flag))) break;
        tc_fence_after();
        const int key0 = j * kTileN;
        if (PAIR && j > 0 && key0 + kTileN - 1 <= warp_lim0) {
          // A tile that every row sees whole, in the middle of a sequence: the
          // row stays in registers and the first part's exponentials use the running
          // maximum while the tile's own is computed (see the chunk kernel).
          uint32_t u[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, u[q]);
          tmem_ld_wait();
          float sv[128];
#pragma unroll
          for (int c = 0; c < 128; ++c) sv[c] = __uint_as_float(u[c >> 5][c & 31]);
          const float2 sl2 = make_float2(sl, sl);
          float2 rs4[4];
          float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int k = 0; k < 4; ++k) rs4[k] = make_float2(0.f, 0.f);
          exps_to_tmem<0, S::KP0, false>(sv, sl2, make_float2(-mb, -mb), rs4, tS);
          float mx8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = sv[k];
#pragma unroll
          for (int c = 8; c + 16 <= 128; c += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], sv[c + 2 * k], sv[c + 2 * k + 1]);
          // (the last step takes four pairs twice, which leaves the maximum unchanged)
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], sv[120 + 2 * (k & 3)], sv[121 + 2 * (k & 3)]);
          const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
          if (raise(mx)) {
            mb = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int k = 0; k < 4; ++k) rs4[k] = make_float2(0.f, 0.f);
            tmem_st_wait();
            // rows whose reference did not move recompute the same values
            exps_to_tmem<0, S::KP0, false>(sv, sl2, make_float2(-mb, -mb), rs4, tS);
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar(S::B_P + x));
          if (S::SPLIT_P) {
            exps_to_tmem<S::KP0, kTileN, false>(sv, sl2, make_float2(-mb, -mb), rs4, tS);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar(S::B_P1 + x));
          }
          const float2 rs2 = fadd2(fadd2(rs4[0], rs4[1]), fadd2(rs4[2], rs4[3]));
          l += rs2.x + rs2.y;
          continue;
        }
        // The first tile and those on the diagonal, in a loop over chunks of 32
        // keys that leaves out the chunks that no row of the warp sees (from
        // `hidden` on; lim rises with the row).  A loop, because this path and the
        // one above, both unrolled, outgrow the instruction cache when every item is
        // a few tiles: 64 prompts of 512 tokens took 303 us, this way 199 us.
        const int hidden = min(4, (warp_lim - key0) / 32 + 1);
        // ---- row maximum
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < hidden; ++c) {
          float s[32];
          load_scores(tS + 32 * c, key0 + 32 * c, lim, s);
          float m4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmax3(s[k], s[4 + k], s[8 + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmax3(m4[k], s[12 + k], s[16 + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmax3(m4[k], s[20 + k], s[24 + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], s[28 + k]);
          mx = fmax3(mx, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        raise(mx);
        // ---- P, over the S columns already read: chunk c's 16 columns of bf16
        // pairs lie at or before its 32 columns of scores
        const float mb = m == -INFINITY ? 0.f : m;
        const float2 sl2 = make_float2(sl, sl), nmb2 = make_float2(-mb, -mb);
        float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
          if (c < hidden) {
            float s[32];
            load_scores(tS + 32 * c, key0 + 32 * c, lim, s);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 e = ffma2(make_float2(s[2 * k], s[2 * k + 1]), sl2, nmb2);
              const float2 pv = make_float2(ex2_approx(e.x), ex2_approx(e.y));
              rs[k & 1] = fadd2(rs[k & 1], pv);
              pk[k] = pack_bf16x2(pv.x, pv.y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) pk[k] = 0u;
          }
          tmem_st16(tS + 16 * c, pk);
          if (c == 3 || (S::SPLIT_P && c == S::KP0 / 32 - 1)) {
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar((S::SPLIT_P && c == 3 ? S::B_P1 : S::B_P) + x));
          }
        }
        l += (rs[0].x + rs[0].y) + (rs[1].x + rs[1].y);
      }
      if (!ok) break;
      mine += n;
      if (!(ok = warp_wait(bar(S::B_O + x), outputs & 1, p.status, abort_flag))) break;
      ++outputs;
      tc_fence_after();
      // The next item's first P V writes O after this group's next P, so after
      // these loads.
      const bool valid = tok < it.len && row < G * T;
      const int hq = it.g * G + row_head;
      // (a row whose scores are all -inf: 0)
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // A thread holds a row, whose direct 16-byte stores would touch 32 lines
      // an instruction (3 us an item).  Each 32 dims are transposed within groups of four lanes
      // first: lane a of a group gets dims 8a .. 8a + 7 of the group's four
      // rows, and four lanes store 64 consecutive bytes of one row.
      const int a = lane & 3;
      uint16_t* dst[4];  // this lane's piece of the group's row k, null for rows that are not stored
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = wq * 32 + (lane & ~3) + k;
        const int t = it.tok0 + x * T + r / G;
        dst[k] = t < it.len && r < G * T
                     ? p.out + (static_cast<int64_t>(it.start + t) * p.heads + it.g * G + r % G) * DV + 8 * a
                     : nullptr;
      }
#pragma unroll 1
      for (int q = 0; q < DV / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * q, o);
        tmem_ld_wait();
        uint32_t w[4][4];  // [piece of 8 dims][word]
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          // (two products an instruction; -0 as the addend leaves them as they are)
          const float2 e = ffma2(make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])),
                                 make_float2(inv, inv), make_float2(-0.f, -0.f));
          w[k >> 2][k & 3] = pack_bf16x2(e.x, e.y);
        }
        transpose4(w, a);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (dst[k]) *reinterpret_cast<uint4*>(dst[k] + 32 * q) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
      }
      if (valid && p.lse) p.lse[static_cast<int64_t>(hq) * p.total + it.start + tok] = m * kLn2 + logf(l);
      tc_fence_before();
    }
  }

  // TMEM is freed once the warps that use it are done (an mbarrier, since the
  // lanes of the low warpgroup come here at different times); see the chunk
  // kernel.
  if (warp >= 4) {
    __syncwarp();
    tc_fence_before();
    if (lane == 0) mbar_arrive(bar(S::B_END));
  } else if ((warp == 1 || (PAIR && warp == 3)) && lane == 0) {
    tc_fence_before();
    mbar_arrive(bar(S::B_END));
  }
  if (warp == 2) {
    __syncwarp();
    // Waits as long as the roles do: each of their waits is bounded.
    while (!mbar_wait_for(bar(S::B_END), 0, 2 * kWaitTimeoutNs + 2 * kCleanupNs) && !*abort_flag) {
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, S::TMEM_COLS);
  }
}

// x / d = x * mul >> shift, with 2^shift at least 2^30 d: exact while x times the excess
// of mul * d over 2^shift, which is below d, is less than 2^shift; that holds for x up to
// 2^30 + 512 and every d up to 1024.
void divide_by(int d, uint64_t* mul, int32_t* shift) {
  *shift = 30;
  while (1 << (*shift - 30) < d) ++*shift;
  *mul = ((1ull << *shift) + d - 1) / d;
}

template <int DQ, int DV, bool PAIR>
cudaError_t launch_prompt_t(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                            PromptParams p, cudaStream_t stream) {
  using S = PShape<DQ, DV, PAIR>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    e = cudaFuncSetAttribute(prompt_attn_kernel<DQ, DV, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  // Items: at most one for each whole tile (pair) of the rows and one partial
  // one for each sequence.
  const int tokens = S::TILES * (kTileM / (p.heads / p.kv_heads));
  const int64_t items = (p.total / tokens + std::min<int64_t>(p.batch, p.total)) * p.kv_heads;
  if (items > INT32_MAX / 2) return cudaErrorInvalidValue;
  p.item_tokens = tokens;
  divide_by(tokens, &p.item_mul, &p.item_shift);
  divide_by(p.kv_heads, &p.head_mul, &p.head_shift);
  return launch_overlapped(prompt_attn_kernel<DQ, DV, PAIR>, dim3(static_cast<unsigned>(items)), S::THREADS, S::SMEM, stream,
                           tm_q, tm_k, tm_v, p);
}

// One query tile a CTA, two CTAs per SM, for short sequences and for few tiles; otherwise
// pairs, which read each key tile half as often but run a tile that has no partner alone.
// The host knows the rows and the number of sequences, not the lengths.
//
// Short: up to 96 rows a sequence, or as many as a tile holds (groups of 1), or 128 at
// 64/64 dims.  One tile a CTA and pairs, us, about 32768 tokens in equal prompts:
//   tokens a prompt          48        64        96       112       128
//   32/8 heads of 128   145 146   119 119   118 139   131 124   117 107
//   16/8                 78 135    67 105    77  77    70  69    63  63
//   64/8                228 271   225 219   224 217   226 237   224 204
//   32/8 heads of 64    107 125    85  97    85 117    98 104    86  89
//   8/8 heads of 128                58 101    46  70              45  54
// and 300 prompts of random lengths, means 64, 96 and 128: 32/8 heads of 128 87 95,
// 143 140, 189 177; 64/8 150 154, 255 238, 341 306; 32/8 of 64 64 80, 101 119, 130 151.
// (96 loses up to 7% for random lengths, less would lose 18% for equal ones.)
// Lengths that are far apart are misjudged, and so are empty sequences and rows of no
// sequence: one prompt of 16384 tokens in 256 slots takes 1954 and 1378.
//
// Few tiles: no more than SMs, of no more than six key tiles.  One prompt of 77, 200, 300,
// 400, 500, 600 tokens (24 to 152 tiles) 7.3 7.9, 9.0 10.0, 10.8 11.8, 12.5 11.9, 12.9 13.4,
// 14.6 14.7, of 650 and 800 17.0 15.4, 19.2 17.0; 64/8 heads of 128, 150 and 300 tokens
// (80, 152 tiles) 9.2 9.8, 11.0 11.7; 8/8, 700 and 1100 (48, 72 tiles) 15.7 16.4, 21.0 19.6;
// 32/8 of 64, 600 tokens 12.3 13.4.
template <int DQ, int DV>
cudaError_t launch_prompt_d(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                            const PromptParams& p, int num_sms, cudaStream_t stream) {
  if constexpr (DQ <= 128) {  // (three stages of 192 dims do not fit half an SM)
    const int64_t tokens = kTileM / (p.heads / p.kv_heads);
    const int64_t tiles = (p.total / tokens + std::min<int64_t>(p.batch, p.total)) * p.kv_heads;
    const int64_t few_rows = DQ + DV <= 128 ? kTileN : std::max<int64_t>(tokens, 96);
    if (p.total <= few_rows * p.batch || (tiles <= num_sms && p.total <= 6 * kTileN))
      return launch_prompt_t<DQ, DV, false>(tm_q, tm_k, tm_v, p, stream);
  }
  return launch_prompt_t<DQ, DV, true>(tm_q, tm_k, tm_v, p, stream);
}

}  // namespace

cudaError_t launch_prompt_attn(int dq, int dv, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, const PromptParams& p, int num_sms, cudaStream_t stream) {
  if (dq == 64 && dv == 64) return launch_prompt_d<64, 64>(tm_q, tm_k, tm_v, p, num_sms, stream);
  if (dq == 64 && dv == 128) return launch_prompt_d<64, 128>(tm_q, tm_k, tm_v, p, num_sms, stream);
  if (dq == 128 && dv == 64) return launch_prompt_d<128, 64>(tm_q, tm_k, tm_v, p, num_sms, stream);
  if (dq == 128 && dv == 128) return launch_prompt_d<128, 128>(tm_q, tm_k, tm_v, p, num_sms, stream);
  if (dq == 192 && dv == 64) return launch_prompt_d<192, 64>(tm_q, tm_k, tm_v, p, num_sms, stream);
  if (dq == 192 && dv == 128) return launch_prompt_d<192, 128>(tm_q, tm_k, tm_v, p, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace vpp
