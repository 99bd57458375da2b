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
// Items.  An item is a pair of query tiles (2T tokens, T = floor(128 / G), times the G
// heads of one kv head) of one sequence.  The sequences are read from
// cu_seqlens on the device.  Sequence b has np_b = ceil(len_b / 2T) pairs, and pair j
// attends to about (j + 1) 2T keys whatever its sequence, so the items are
// ordered by j, largest first: F(j) = sum_b max(0, np_b - j) counts those of
// pair index >= j; item i has the largest j with F(j) > i, found by bisection, and
// belongs to the (i - F(j + 1))-th sequence with np_b > j.
//
// Persistent CTAs.  One CTA per SM takes every grid-th item, the order
// reversed in every other round, which evens out the rounds' sums.  The chunk
// kernel's one-item CTAs cost about 8 us each besides their keys (launch, TMEM, first
// loads, drain, output), most of the time of short prompts.  Here the next item's
// Q and K/V copies and its first Q K^T run while the last softmax and the output
// of the current one do.
//
//   warp 0      TMA producer (Q of the item, then K and V tiles, ring of 16 KB slots)
//   warp 1, 3   MMA issuers of query tiles A and B, taking turns
//   warp 2      TMEM; finds the items ahead of their use and hands them out
//               through four shared-memory entries; zeroes the V rows of other
//               sequences in an item's last tile (P = 0 times whatever they hold
//               must stay 0; their K rows are masked before the softmax)
//   warps 4-7, 8-11   softmax and output of tiles A and B
//
// The two tiles of a pair may need different numbers of key tiles (nA <= nB; B is
// absent when the sequence ends in A), and each runs its own number.
//
// Bound by the tensor core for long prompts, by the chain of one item for short ones.
#include <algorithm>

#include "chunk_attn_impl.cuh"
#include "prompt_attn.cuh"

namespace vpp {
namespace {

using namespace attn_detail;

constexpr int kEntries = 4;  // items handed out ahead

struct Item {
  int start, len;  // the sequence's rows
  int tok0;        // first token of tile A
  int g;           // kv head
  int na, nb;      // key tiles of A and of B (nb = 0: no B)
  int pad[2];
};

template <int DQ, int DV>
struct PShape : Shape<DQ, DV, false> {
  using S = Shape<DQ, DV, false>;
  static constexpr int B_Q = 0, B_QE = 1, B_S = 2, B_P = 4, B_P1 = 6, B_O = 8, B_FINAL = 10, B_END = 12, B_IF = 13,
                       B_IE = B_IF + kEntries, B_FULL = B_IE + kEntries, B_EMPTY = B_FULL + S::NB,
                       B_TMP = B_EMPTY + S::NB, NBARS = B_TMP + S::NB;
  static constexpr int SMEM = 1024 + S::QBYTES + S::NSLOT * kSubTileBytes + kEntries * 32 + NBARS * 8 + 16;
  static_assert(SMEM <= kSmemLimit, "shared memory budget");
};

// The work list, by one warp: a sequence per lane, more in further rounds.
struct Finder {
  const PromptParams& p;
  int T2, lane, np0, hi;  // hi: F(hi) <= every item still to come
  __device__ __forceinline__ Finder(const PromptParams& p_, int T2_) : p(p_), T2(T2_) {
    lane = threadIdx.x & 31;
    np0 = pairs(lane);
    hi = static_cast<int>((p.total + T2 - 1) / T2);
  }
  __device__ __forceinline__ int pairs(int b) const {
    if (b >= p.batch) return 0;
    const int lo = __ldg(p.cu + b), end = __ldg(p.cu + b + 1);
    if (lo < 0 || end < lo || end > p.total) {
      if (blockIdx.x == 0) record_status(p.status, kStatusInvalid);
      return 0;
    }
    return (end - lo + T2 - 1) / T2;
  }
  // F(j): pairs of index >= j over all sequences.
  __device__ __forceinline__ int count(int j) const {
    int s = max(0, np0 - j);
    for (int b = lane + 32; b < p.batch; b += 32) s += max(0, pairs(b) - j);
    return __reduce_add_sync(0xffffffffu, s);
  }
  // Item i (items are asked for in increasing order, so j only falls).
  __device__ __forceinline__ void find(int i, int* b_out, int* j_out) {
    int j = 0, top = hi;  // F(j) > i >= F(top)
    while (top - j > 1) {
      const int mid = (j + top) >> 1;
      if (count(mid) > i) j = mid; else top = mid;
    }
    hi = top;
    int rank = i - count(j + 1);
    *b_out = -1;  // (none: only when the ranges overlap and the counts overflow)
    for (int base = 0; base < p.batch; base += 32) {
      const bool in = (base == 0 ? np0 : pairs(base + lane)) > j;
      const uint32_t mask = __ballot_sync(0xffffffffu, in);
      const int n = __popc(mask);
      if (rank < n) {
        const bool mine = in && __popc(mask & ((1u << lane) - 1u)) == rank;
        *b_out = base + __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        *j_out = j;
        return;
      }
      rank -= n;
    }
  }
};

template <int DQ, int DV>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PromptParams p) {
  using S = PShape<DQ, DV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + S::QBYTES;
  Item* entries = reinterpret_cast<Item*>(sRing + S::NSLOT * kSubTileBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(entries + kEntries);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + S::NBARS);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
  volatile int* turn = reinterpret_cast<volatile int*>(tmem_slot + 2);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.heads / p.kv_heads;
  const int T = kTileM / G;  // tokens per query tile

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    *turn = 0;
    mbar_init(bar(S::B_Q), 1);
    mbar_init(bar(S::B_QE), 2);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(S::B_S + x), 1);
      mbar_init(bar(S::B_P + x), 128);
      mbar_init(bar(S::B_P1 + x), 128);
      mbar_init(bar(S::B_O + x), 1);
      mbar_init(bar(S::B_FINAL + x), 1);
    }
    mbar_init(bar(S::B_END), 10);  // the 8 softmax warps and the 2 MMA issuers
    for (int i = 0; i < kEntries; ++i) {
      mbar_init(bar(S::B_IF + i), 1);
      mbar_init(bar(S::B_IE + i), 11);  // producer, 2 issuers, 8 softmax warps
    }
    for (int i = 0; i < S::NB; ++i) {
      mbar_init(bar(S::B_FULL + i), 1);
      mbar_init(bar(S::B_EMPTY + i), 2);  // released by both MMA issuers
      mbar_init(bar(S::B_TMP + i), 1);
    }
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  // Item i of this CTA, as one thread (producer, issuer) reads it.
  auto take = [&](int i, Item* it) {
    if (!mbar_wait(bar(S::B_IF + i % kEntries), (i / kEntries) & 1, p.status, abort_flag)) return false;
    *it = entries[i % kEntries];
    mbar_arrive(bar(S::B_IE + i % kEntries));
    return it->len > 0;
  };

  if (warp < 4) {
    regs_dec<kRegsLow>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA producer
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      bool ok = true;
      int base = 0;    // tile pairs (K and V) of the items before
      int issued = 0;  // tiles whose loads were started
      int rq = 0;      // next tile whose release has not been observed
      uint32_t tmp_phase = 0u, tmp_last = 0u;  // parity of B_TMP's next use; tiles that landed there last
      int n_items = 0;
      Item it;
      for (int i = 0; ok && take(i, &it); ++i) {
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
      Finder finder(p, 2 * T);
      const int total =
          static_cast<int>(min(static_cast<int64_t>(INT32_MAX / 2), static_cast<int64_t>(finder.count(0)) * p.kv_heads));
      int round = 0, published = 0;
      bool done = false, ok = true;
      auto publish = [&]() {
        if (done || !ok) return;
        const int grid = gridDim.x, c = blockIdx.x;
        int idx = round * grid + ((round & 1) ? grid - 1 - c : c);
        if (idx >= total) {  // nothing for this CTA in the last round, or past it
          done = true;
        }
        ++round;
        Item it{0, 0, 0, 0, 0, 0, {0, 0}};
        if (!done) {
          int b, j;
          const int item = idx / p.kv_heads;
          finder.find(item, &b, &j);
          done = b < 0;
          b = max(b, 0);
          it.start = __ldg(p.cu + b);
          it.len = __ldg(p.cu + b + 1) - it.start;
          it.tok0 = j * 2 * T;
          it.g = idx - item * p.kv_heads;
          it.na = (min(it.tok0 + T, it.len) + kTileN - 1) / kTileN;
          if (done) it.len = 0;
          it.nb = it.tok0 + T < it.len ? (min(it.tok0 + 2 * T, it.len) + kTileN - 1) / kTileN : 0;
        }
        const int e = published % kEntries;
        if (published >= kEntries &&
            !(ok = warp_wait(bar(S::B_IE + e), (published / kEntries - 1) & 1, p.status, abort_flag)))
          return;
        if (lane == 0) {
          entries[e] = it;
          mbar_arrive(bar(S::B_IF + e));
        }
        __syncwarp();
        ++published;
      };
      publish();
      publish();
      int base = 0;
      uint32_t tmp_phase = 0u;
      for (int i = 0; ok; ++i) {
        publish();  // item i + 2
        if (!ok || i >= published) break;
        const Item it = entries[i % kEntries];  // (overwritten by item i + 4 at the earliest)
        if (it.len == 0) break;
        const int n = max(it.na, it.nb);
        const int t = 2 * (base + n) - 1;
        const int r0 = it.len - (n - 1) * kTileN;
        if (r0 < kTileN) {
          const int tb = t % S::NB;
          if (!(ok = warp_wait(bar(S::B_TMP + tb), (tmp_phase >> tb) & 1u, p.status, abort_flag))) break;
          tmp_phase ^= 1u << tb;
          const int pos = S::tile_pos(t);
          for (int u = r0 * 8 + lane; u < kTileN * 8; u += 32)  // 16-byte units of rows r0 .. 127
#pragma unroll
            for (int c = 0; c < S::NVC; ++c)
              *reinterpret_cast<uint4*>(sRing + ((pos + c) % S::NSLOT) * kSubTileBytes + u * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(S::B_FULL + tb));
        }
        base += n;
      }
    } else if ((warp == 1 || warp == 3) && lane == 0) {
      // ---------------------------------------------------- MMA issuer
      const int x = warp == 1 ? 0 : 1;
      const uint64_t dq0 = sdesc_sw128(smem_u32(sQ + x * S::NQC * kSubTileBytes), 16, 1024);
      const uint64_t dk0 = sdesc_sw128(smem_u32(sRing), 16, 1024);             // K-major
      const uint64_t dv0 = sdesc_sw128(smem_u32(sRing), kSubTileBytes, 1024);  // MN-major
      constexpr uint32_t kSub16 = kSubTileBytes >> 4;
      const uint32_t tS = tbase + x * kTileN;
      const uint32_t tO = tbase + 2 * kTileN + x * DV;
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
            // Take the turn: a tight spin on the shared counter (the abort flag
            // and the time limit are checked every 256 polls).
            if (*turn != my_turn) {
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
              const bool adjacent = S::NVC == 1 || vslot + S::NVC <= S::NSLOT;
              auto pv_steps = [&](int k0, int k1) {
                if (adjacent) {
                  const uint64_t vb = dv0 + vslot * kSub16;
#pragma unroll
                  for (int k = k0; k < k1; ++k)
                    umma_ts(tO, tS + 8 * k, vb + k * (2048 >> 4), S::IDESC_PV, (j > 1 || k > 0) ? 1u : 0u);
                } else {
#pragma unroll
                  for (int k = k0; k < k1; ++k)
#pragma unroll
                    for (int h = 0; h < S::NVC; ++h) {
                      const int vs = vslot + h < S::NSLOT ? vslot + h : vslot + h - S::NSLOT;
                      umma_ts(tO + 64 * h, tS + 8 * k, dv0 + vs * kSub16 + k * (2048 >> 4), S::IDESC_PV64,
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
                  if (c == S::NQC - 1 && k == 0) *turn = my_turn + 1;
                  umma_ss(tS, dq0 + c * kSub16 + 2 * k, kb + 2 * k, S::IDESC_QK, (c | k) ? 1u : 0u);
                }
              }
              umma_commit(bar(S::B_S + x));
              umma_commit(bar(S::B_EMPTY + tk % S::NB));
              if (j >= ny) mbar_arrive(bar(S::B_EMPTY + tk % S::NB));  // the partner does not read this tile
              if (j == nx - 1) {
                umma_commit(bar(S::B_QE));
                if (ny == 0) mbar_arrive(bar(S::B_QE));
              }
            } else {
              *turn = my_turn + 1;
            }
            if (j > 0) {
              if (!S::EARLY_V) umma_commit(bar(S::B_EMPTY + tv % S::NB));
              if (j - 1 >= ny) mbar_arrive(bar(S::B_EMPTY + tv % S::NB));
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
    const uint32_t tO = lane_base + 2 * kTileN + x * DV;
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
      float m = -INFINITY;  // running max of score * scale * log2(e)
      float l = 0.f;        // running denominator, relative to 2^m
      for (int j = 0; j < n; ++j) {
        if (!(ok = warp_wait(bar(S::B_S + x), (mine + j) & 1, p.status, abort_flag))) break;
        tc_fence_after();
        uint32_t u[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, u[q]);
        tmem_ld_wait();
        float sv[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) sv[c] = __uint_as_float(u[c >> 5][c & 31]);
        const int key0 = j * kTileN;
        if (key0 + kTileN - 1 > lim) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (key0 + c > lim) sv[c] = -INFINITY;
        }
        // Row max: eight independent chains of 3-input max, then a tree (the
        // last step takes four pairs twice, which leaves the maximum unchanged).
        auto row_max = [&]() {
          float mx8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = sv[k];
#pragma unroll
          for (int c = 8; c + 16 <= 128; c += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], sv[c + 2 * k], sv[c + 2 * k + 1]);
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], sv[120 + 2 * (k & 3)], sv[121 + 2 * (k & 3)]);
          return fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        };
        const float2 sl2 = make_float2(sl, sl);
        float2 rs4[4];
        auto part = [&](auto k0, auto k1, float mref) {
          const float mb = (mref == -INFINITY) ? 0.f : mref;
          const float2 nmb2 = make_float2(-mb, -mb);
          exps_to_tmem<decltype(k0)::value, decltype(k1)::value, false>(sv, sl2, nmb2, rs4, tS);
        };
        using K_0 = std::integral_constant<int, 0>;
        using K_P0 = std::integral_constant<int, S::KP0>;
        using K_N = std::integral_constant<int, kTileN>;
#pragma unroll
        for (int k = 0; k < 4; ++k) rs4[k] = make_float2(0.f, 0.f);
        if (j == 0) {
          m = row_max() * sl;
          part(K_0{}, K_P0{}, m);
        } else {
          // The first part's exponentials use the running max right away; only
          // when the tile's own max has grown by more than 2^8 are O, the
          // denominator and that part redone (exact either way: numerator and
          // denominator share the reference m).
          part(K_0{}, K_P0{}, m);
          const float m_new = fmaxf(m, row_max() * sl);
          const bool need = m_new > m + kRescaleThreshold;
          if (__any_sync(0xffffffffu, need)) {
            // O is idle here: PV(x, j-1) completed before S(x, j) was
            // committed, and PV(x, j) waits for this group's P.
            const float f = need ? ex2_approx(m - m_new) : 1.f;
            if (need) {
              l *= f;
              m = m_new;
            }
            tmem_st_wait();
#pragma unroll
            for (int q = 0; q < DV / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * q, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st32(tO + 32 * q, o);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) rs4[k] = make_float2(0.f, 0.f);
            part(K_0{}, K_P0{}, m);  // rows whose m did not move recompute the same values
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(S::B_P + x));
        if (S::SPLIT_P) {
          part(K_P0{}, K_N{}, m);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar(S::B_P1 + x));
        }
        const float2 rs2 = fadd2(fadd2(rs4[0], rs4[1]), fadd2(rs4[2], rs4[3]));
        l += rs2.x + rs2.y;
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
      const float inv = 1.f / l;
      uint16_t* orow = p.out + (static_cast<int64_t>(it.start + tok) * p.heads + hq) * DV;
#pragma unroll
      for (int q = 0; q < DV / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * q, o);
        tmem_ld_wait();
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          pk[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
        if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(orow + 32 * q);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
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
  } else if ((warp == 1 || warp == 3) && lane == 0) {
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
    tmem_dealloc(tbase, 512);
  }
}

template <int DQ, int DV>
cudaError_t launch_prompt_t(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                            const PromptParams& p, int grid, cudaStream_t stream) {
  constexpr int smem = PShape<DQ, DV>::SMEM;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool configured[64] = {};
  if (dev < 64 && !configured[dev]) {
    e = cudaFuncSetAttribute(prompt_attn_kernel<DQ, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  prompt_attn_kernel<DQ, DV><<<grid, kAttnThreads, smem, stream>>>(tm_q, tm_k, tm_v, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_attn(int dq, int dv, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, const PromptParams& p, int64_t items, int num_sms,
                               cudaStream_t stream) {
  const int grid = static_cast<int>(std::min<int64_t>(items * p.kv_heads, num_sms));
  if (dq == 64 && dv == 64) return launch_prompt_t<64, 64>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 64 && dv == 128) return launch_prompt_t<64, 128>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 128 && dv == 64) return launch_prompt_t<128, 64>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 128 && dv == 128) return launch_prompt_t<128, 128>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 192 && dv == 64) return launch_prompt_t<192, 64>(tm_q, tm_k, tm_v, p, grid, stream);
  if (dq == 192 && dv == 128) return launch_prompt_t<192, 128>(tm_q, tm_k, tm_v, p, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace vpp
