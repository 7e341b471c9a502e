// attn_fwd_mod_tc.cu -- bf16 attention forward with modified scores on the
// 5th-generation tensor cores.
//
// O = P V with P the softmax of the scores of score_mod.cuh over the keys each
// row sees (mask.cuh), plus the row log-sum-exp; layouts as the plain forward
// (attn_fwd_tc.cu): head-sharded, query head j of a rank reads kv-head
// j / (hp / kvp).
//
// The pipeline is the plain forward's: one CTA per pair of 128-query tiles (A,
// B) of one head, a TMA warp that feeds (V_e, K_{e+1}) pairs through a two-entry
// ring, one issuing thread in the order S_A S_B | PV_A S_A PV_B S_B | .., P
// read from TMEM as the A operand.  The key tiles are the hull of what the
// pair's rows see, not [0, n); a pair that sees nothing writes zeros and -inf
// and leaves.  With a bias the tiles run from the last key to the first: there
// the diagonal, where the bias is 0, comes first and sets the rows' references.
//
// The chain S -> softmax -> PV of a tile is what bounds these kernels, so the
// softmax has two forms:
//   narrow (the plain forward's): one warpgroup a tile, a thread holds a whole
//     row's 128 scores; the row's reference (the offset of its exponents) is set
//     on the first tile in which it sees a key and moved when a sum of P passes
//     2^16.
//   wide, for capped scores without a bias: these lie in [-cap, cap], so with
//     cap log2(e) <= 80 every P = 2^x is a normal number without any reference
//     (x within +-80, sums below 2^80 S), and the threads of a row need not
//     agree on one.  Two warpgroups share a tile, 64 scores a thread, taken 16
//     at a time; they meet once, when the sums are added at the end.
// 32K tokens x 8 heads of 128, causal, capped at 50: narrow 1914 us, wide
// 1660 us (0.68 of the measured bf16 rate); the plain forward there 1340 us.
//
// Documents make items of a few key tiles, where a block's start (barriers,
// tensor memory, Q and the first K from memory, the first scores) and its
// epilogue cost as much as its steps.  So blocks go on with items of blocks that
// have not started (work_items.cuh): the next item's Q, K and V are loaded and
// its first scores formed while the last steps and the epilogue of this one run,
// and its rows' key intervals arrive meanwhile.  8K tokens x 32 heads of 128 in
// eight equal documents, mask alone: 109 -> 76 us (by now 72), capped at 50, which
// no score came near, 134 -> 97; heads of 64 91 -> 66 and 111 -> 90 (64, 86).  In
// documents of random lengths about 1024, a cap of 20 reached: 185-205 us by where
// they lie.  In a step that needs masking, 16-key chunks that no row of the
// warp sees are skipped.
// Every wait is bounded (2 s), as in the plain forward.
#include <cuda_bf16.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "check.cuh"
#include "internal.h"
#include "score_mod.cuh"
#include "sm100.cuh"
#include "tmap.h"
#include "work_items.cuh"

namespace ulysses {
namespace {

using namespace sm100;
using dev::bits_of;
using dev::get_item;
using dev::Item;
using dev::put_item;
using dev::warp_wait;

constexpr int BM = 128;  // query rows per tile (two tiles per CTA)
constexpr int BN = 128;  // keys per tile
// Warps: the softmax warpgroups (2, wide: 4), then one of TMA, MMA and 2 idle
// warps.  Registers: narrow launches 384 threads x 168 and splits them 216 / 64,
// wide 640 x 96 and 104 / 64 (each warpgroup's threads times its limit add up
// to no more than the launch's).
template <bool kWide>
struct Roles {
  static constexpr int kSoftmax = kWide ? 16 : 8;
  static constexpr int kTmaWarp = kSoftmax, kMmaWarp = kSoftmax + 1;
  static constexpr int kThreads = 32 * (kSoftmax + 4);
  static constexpr int kRowThreads = kWide ? 2 : 1;  // threads of a row
  static constexpr uint32_t kRegsProducer = 64, kRegsSoftmax = kWide ? 104 : 216;
  static_assert(128 * kRegsProducer + 32 * kSoftmax * kRegsSoftmax <= (uint32_t)kThreads * (kWide ? 96 : 168),
                "register split over budget");
};
constexpr int kAhead = 3;  // ring entries before its end at which an item's successor is asked for
constexpr int kSlots = 2;  // K/V ring entries: entry e holds V_e and K_{e+1}
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kChunkBytes = 128 * 128;  // 128 rows x 128 bytes (64 bf16)

template <int D>
struct Layout {
  static constexpr uint32_t kTile = 128u * D * 2;   // one 128-row tile of Q, K or V
  static constexpr uint32_t kEntry = 2 * kTile;     // V_e, then K_{e+1}
  static constexpr uint32_t kQ = 0;                 // Q_A, Q_B
  static constexpr uint32_t kK0 = kQ + 2 * kTile;   // K_0
  static constexpr uint32_t kKV = kK0 + kTile;      // ring of kSlots entries
  // wide: float [2 tiles][2 halves][128 rows], the sums of the rounded P, and int16
  // [2 tiles][128 rows], how much of half 1's is rounding, in steps of 2^-22
  static constexpr uint32_t kRed = kKV + kSlots * kEntry, kOff = kRed + 2 * 2 * 128 * 4;
  static constexpr uint32_t kBar = kOff + 2 * 128 * 2;
  static constexpr uint32_t kUsed = kBar + 288;
  // room to align the base to 1024 bytes where it fits
  static constexpr uint32_t kAlloc = kUsed + 1024 <= 232448 ? kUsed + 1024 : 232448;
  static_assert(kUsed <= 232448, "shared memory");
};

// Barrier slots (byte offsets inside the barrier block).
enum : uint32_t {
  kBarQFull = 0,
  kBarKVFull = 8,                         // [kSlots]
  kBarKVEmpty = kBarKVFull + 8 * kSlots,  // [kSlots]
  kBarSFull = kBarKVEmpty + 8 * kSlots,   // [2] A, B
  kBarPFull = kBarSFull + 16,             // [2] A, B (every softmax thread of the tile)
  kBarODone = kBarPFull + 16,             // [2] A, B
  kBarSum = kBarODone + 16,               // [2] wide: both halves' sums are in shared memory
  kBarRead = kBarSum + 16,                // [2] wide: and have been read again
  kBarQEmpty = kBarRead + 16,             // the item's last scores have been formed: Q and K_0 are free
  kBarTaken = kBarQEmpty + 8,             // the answer on a block to take over is in kTakenSlot
  kBarItem = kBarTaken + 8,               // [2] item n's facts are in slot n & 1 of kItemSlot
  kBarItemEmpty = kBarItem + 16,          // [2] every warp is through with that item
  kBarDrain = kBarItemEmpty + 16,
  kTmemSlot = kBarDrain + 8,
  kAbortSlot = kTmemSlot + 4,
  kTakenSlot = (kAbortSlot + 4 + 15) / 16 * 16,
  kItemSlot = kTakenSlot + 16  // [2] x 32 bytes
};
constexpr uint32_t kBarBytes = 288;
static_assert(kItemSlot + 64 <= kBarBytes, "barrier block");

struct FwdParams {
  int B, S, hp, kvp, group, causal, n_pairs;
  int head_group;  // heads per CTA group (grouped_order)
  int Pu, Cs;      // ranks of a ring position, tokens of its chunk (plain Ulysses: P, S)
  float scale_log2;
  __nv_bfloat16 *o;      // [P][B][Cs][hp][D]
  float *lse;            // [P][B][hp][Cs]
  int o_by32;            // o lies on a 32-byte boundary
  long long o_n, lse_n;  // their elements (range checks of a checked build)
  uint32_t *status;
  dev::ScoreMod mod;
};

// TMA coordinates (row, rank * B + batch) of a head's 128-row tiles, walked in
// position order either way: the tile at position pos lies in ring position
// pos / Cs, row pos % Cs, of group member r's buffers.
struct TileWalk {
  int row, outer, period, step, left;
  __device__ __forceinline__ TileWalk(const FwdParams &p, int rb, int pos) {
    period = p.Cs, step = p.Pu * p.B;
    const int last = (p.S - 1) / period, c = (pos < p.S ? pos : p.S - 1) / period;
    row = pos - c * period;  // (past the sequence end: rows out of range, read as zeros)
    outer = c * step + rb;
    left = last - c;
  }
  template <bool kBack>
  __device__ __forceinline__ void next() {
    if constexpr (kBack) {
      row -= 128;
      if (row < 0) row += period, outer -= step;
    } else {
      row += 128;
      if (row >= period && left > 0) row -= period, outer += step, --left;
    }
  }
};

// The item of a block: a pair of query tiles (`tile`) of one head, key tiles
// [t0, t0 + nA) of tile A, [t0, t0 + nB) of tile B, nA <= nB.
template <bool kBack>
__device__ __forceinline__ Item item_of(const FwdParams &p, int block) {
  Item it;
  const dev::HeadTile ht = dev::grouped_order(block, p.Pu * p.B * p.hp, p.n_pairs, p.head_group);
  it.tile = p.n_pairs - 1 - ht.rank;  // longest causal pairs first
  it.j = ht.head % p.hp;
  it.rb = ht.head / p.hp;
  const int n_kt = (p.S + BN - 1) / BN, m = 2 * it.tile;
  it.t0 = 0;
  if (p.mod.mask.ranges) {
    const long long at = (long long)(it.rb % p.B) * n_kt + m;
    const int4 ta = dev::tile_at(p.mod.mask, at, p.status);
    const int4 tb = m + 1 < n_kt ? dev::tile_at(p.mod.mask, at + 1, p.status) : make_int4(INT_MAX, 0, 0, 0);
    it.t0 = min(ta.x, tb.x) / BN;  // (INT_MAX: nothing is seen, nB is 0 below)
    const int endA = (ta.y + BN - 1) / BN, endB = (tb.y + BN - 1) / BN;
    it.nB = max(max(endA, endB) - it.t0, 0);
    it.nA = min(max(endA - it.t0, 1), it.nB);
  } else {
    it.nA = p.causal ? min(m + 1, n_kt) : n_kt;
    it.nB = p.causal ? min(m + 2, n_kt) : n_kt;
  }
  if constexpr (kBack) it.nA = it.nB;  // (A's own last tile, then, is its second)
  return it;
}

__device__ __forceinline__ uint32_t ring_slot(int e) { return (uint32_t)(e % kSlots); }
__device__ __forceinline__ uint32_t ring_parity(int e) { return (uint32_t)((e / kSlots) & 1); }

template <int D, int kMod, bool kWide>
__global__ void __launch_bounds__(Roles<kWide>::kThreads, 1)
    attn_fwd_mod_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const FwdParams p) {
  using L = Layout<D>;
  using W = Roles<kWide>;
  constexpr int kChunks = D / 64;  // 128-byte swizzle chunks per row
  constexpr int kSoftmax = W::kSoftmax, kTmaWarp = W::kTmaWarp, kMmaWarp = W::kMmaWarp;
  constexpr bool kBack = (kMod & kModBias) != 0;  // key tiles from the last to the first
  constexpr bool kCap = (kMod & kModCap) != 0, kBias = (kMod & kModBias) != 0;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t *smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const uint32_t sQ = sb + L::kQ, sK0 = sb + L::kK0, sKV = sb + L::kKV;
  const uint32_t bar = sb + L::kBar;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kBar + kAbortSlot);
  const volatile uint32_t *gst = p.status;
  if (*gst & (ULYSSES_STATUS_FWD_TIMEOUT | ULYSSES_STATUS_BWD_TIMEOUT)) return;
  if (!dev::mask_matches(p.mod.mask)) {
    if (threadIdx.x == 0) atomicOr(p.status, (uint32_t)ULYSSES_STATUS_MASK);
    return;
  }
  if (pad + L::kUsed > L::kAlloc) {  // uniform over the block: nobody has touched a barrier yet
    if (threadIdx.x == 0) atomicOr(p.status, (uint32_t)ULYSSES_STATUS_SMEM_ALIGN);
    return;
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar + kBarQFull, 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar + kBarKVFull + 8 * i, 1);
      mbar_init(bar + kBarKVEmpty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + kBarSFull + 8 * i, 1);
      mbar_init(bar + kBarPFull + 8 * i, 128 * W::kRowThreads);
      mbar_init(bar + kBarODone + 8 * i, 1);
      mbar_init(bar + kBarSum + 8 * i, 256);
      mbar_init(bar + kBarRead + 8 * i, 256);
      mbar_init(bar + kBarItem + 8 * i, 1);
      mbar_init(bar + kBarItemEmpty + 8 * i, kSoftmax + 1);
    }
    mbar_init(bar + kBarQEmpty, 1);
    mbar_init(bar + kBarTaken, 1);
    mbar_init(bar + kBarDrain, 1);
    *abort_flag = 0;
    put_item(bar + kItemSlot, item_of<kBack>(p, (int)blockIdx.x));
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(bar + kTmemSlot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kBar + kTmemSlot);

  // Key tile of step t; the facts of this CTA's n-th item (from the second on,
  // once kBarItem says so).
  auto tile_of = [](const Item &it, int t) { return kBack ? it.t0 + it.nB - 1 - t : it.t0 + t; };
  auto item_slot = [&](int n) { return bar + kItemSlot + 32 * (n & 1); };
  auto item_parity = [](int n) { return (uint32_t)(((n - 1) >> 1) & 1); };

  if (warp >= kSoftmax) {
    regs_dec<W::kRegsProducer>();
    if (warp == kTmaWarp) {
      if (lane == 0) {
        // ---------------------------------------------------------- producer
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        int issued = -1, n_live = 0;  // the last ring entry filled; items with keys so far
        bool ok = true;
        Item it = get_item(item_slot(0)), next;
        // Takes over a block that has not started as the n-th item (n >= 1), and
        // asks for what it reads first.  (The answer is waited for in any case: it
        // lands in this CTA's shared memory.)
        auto take = [&](int n) -> bool {
          if (n > 1 && !mbar_wait_bounded(bar + kBarItemEmpty + 8 * (n & 1), ((n - 2) >> 1) & 1, abort_flag, gst))
            return false;
          mbar_arrive_expect_tx(bar + kBarTaken, 16);
          dev::take_block(bar + kTakenSlot, bar + kBarTaken);
          volatile int never = 0;
          if (!mbar_wait_bounded(bar + kBarTaken, (n - 1) & 1, &never, nullptr)) {
            *abort_flag = 1;
            return false;
          }
          const int block = dev::taken_block(bar + kTakenSlot);
          if (block >= 0) {
            next = item_of<kBack>(p, block);
          } else {
            next.tile = -1;
          }
          put_item(item_slot(n), next);
          mbar_arrive(bar + kBarItem + 8 * (n & 1));
          if (block >= 0 && next.nB > 0) {
            TileWalk tq(p, next.rb, next.tile * 2 * BM);
            for (int x = 0; x < 2; ++x, tq.next<false>())
              for (int c = 0; c < kChunks; ++c) tma_prefetch_4d(&tmQ, c * 64, next.j, tq.row, tq.outer);
            const TileWalk tv(p, next.rb, tile_of(next, 0) * BN);
            for (int c = 0; c < kChunks; ++c) {
              tma_prefetch_4d(&tmK, c * 64, next.j / p.group, tv.row, tv.outer);
              tma_prefetch_4d(&tmV, c * 64, next.j / p.group, tv.row, tv.outer);
            }
          }
          return true;
        };
        for (int n = 0;; ++n) {
          if (it.nB > 0) {
            // Q_A, Q_B and K_0 on one barrier, once the item before has formed its last scores
            if (n_live > 0 && !(ok = mbar_wait_bounded(bar + kBarQEmpty, (n_live - 1) & 1, abort_flag, gst))) break;
            mbar_arrive_expect_tx(bar + kBarQFull, 3 * L::kTile);
            const int kl = it.j / p.group;
            TileWalk tv(p, it.rb, tile_of(it, 0) * BN);  // step t's key tile (K_t, V_t)
            for (int c = 0; c < kChunks; ++c)
              tma_load_4d(sK0 + c * kChunkBytes, &tmK, bar + kBarQFull, c * 64, kl, tv.row, tv.outer);
            TileWalk tq(p, it.rb, it.tile * 2 * BM);
            for (int x = 0; x < 2; ++x, tq.next<false>())
              for (int c = 0; c < kChunks; ++c)
                tma_load_4d(sQ + x * L::kTile + c * kChunkBytes, &tmQ, bar + kBarQFull, c * 64, it.j, tq.row, tq.outer);
            ++n_live;
            // an entry is V_t and (when tile B goes on) K_{t+1}: what key tile t's two bursts read
            for (int t = 0; t < it.nB; ++t) {
              const int e = issued + 1;
              const uint32_t slot = ring_slot(e), full = bar + kBarKVFull + 8 * slot;
              if (!(ok = mbar_wait_bounded(bar + kBarKVEmpty + 8 * slot, ring_parity(e) ^ 1, abort_flag, gst))) break;
              const bool has_k = t + 1 < it.nB;
              mbar_arrive_expect_tx(full, (has_k ? 2u : 1u) * L::kTile);
              const uint32_t dst = sKV + slot * L::kEntry;
              for (int c = 0; c < kChunks; ++c)
                tma_load_4d(dst + c * kChunkBytes, &tmV, full, c * 64, kl, tv.row, tv.outer);
              tv.next<kBack>();
              if (has_k)
                for (int c = 0; c < kChunks; ++c)
                  tma_load_4d(dst + L::kTile + c * kChunkBytes, &tmK, full, c * 64, kl, tv.row, tv.outer);
              issued = e;
              if (t == max(it.nB - kAhead, 0) && !(ok = take(n + 1))) break;
            }
            if (!ok) break;
          } else if (!(ok = take(n + 1))) {
            break;
          }
          if (next.tile < 0) break;
          it = next;
        }
        if (*abort_flag) {
          // Let the copies already in flight land before the CTA goes away.
          volatile int never = 0;
          if (n_live > 0) mbar_wait_bounded(bar + kBarQFull, (n_live - 1) & 1, &never, nullptr, 500000000ull);
          for (int e = issued - (kSlots - 1); e <= issued; ++e)
            if (e >= 0)
              mbar_wait_bounded(bar + kBarKVFull + 8 * ring_slot(e), ring_parity(e), &never, nullptr, 500000000ull);
        }
      }
    } else if (warp == kMmaWarp) {
      if (lane == 0) {
        // -------------------------------------------------------------- MMA
        constexpr uint32_t idS = idesc_bf16_f32(BM, BN, 0, 0);  // Q, K both K-major
        constexpr uint32_t idPV = idesc_bf16_f32(BM, D, 0, 1);  // P (TMEM), V MN-major
        int e0 = 0, doneA = 0;  // ring entries (and tile B's steps), tile A's steps of the items before
        // S_x(t) = Q_x K_t^T (K_t has landed: the caller waited for it).
        // (The descriptors are one addition each from a base that is formed here:
        // kept for the whole kernel, all of them spilled to memory that each item
        // read again.  Mask alone, those documents: 107 -> 78 us.)
        auto issue_s = [&](int x, int t) {
          uint64_t q = smem_desc_sw128(sQ + x * L::kTile, 16, 1024);
          uint64_t k = smem_desc_sw128(t == 0 ? sK0 : sKV + ring_slot(e0 + t - 1) * L::kEntry + L::kTile, 16, 1024);
          asm volatile("" : "+l"(q), "+l"(k));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t koff = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
            mma_bf16_ss(tmem + x * BN, q + koff, k + koff, idS, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar + kBarSFull + 8 * x);
        };
        // O_x += P_x(t) V_t (P_x(t) published and V_t landed: the caller waited).
        auto issue_pv = [&](int x, int t) {
          uint64_t v = smem_desc_sw128(sKV + ring_slot(e0 + t) * L::kEntry, kChunkBytes, 1024);
          asm volatile("" : "+l"(v));
          // keys 16kk..16kk+15 of P_X: columns 8kk.. of S_X; wide: each half's P lies over
          // the first half of its own scores
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            const uint32_t ac = x * BN + (kWide && kk >= 4 ? 64 + (kk - 4) * 8 : kk * 8);
            mma_bf16_ts(tmem + 2 * BN + x * D, tmem + ac, v + (kk * 16 * 128 >> 4), idPV,
                        (t > 0 || kk > 0) ? 1u : 0u);
          }
        };
        bool ok = true;
        int n_live = 0;
        Item it = get_item(item_slot(0));
        for (int n = 0; it.tile >= 0; ++n) {
          if (it.nB > 0) {
            const int nA = it.nA, nB = it.nB;
            if (!(ok = mbar_wait_bounded(bar + kBarQFull, n_live & 1, abort_flag, gst))) break;
            ++n_live;
            // (The tensor core works in order: the item before has read its last P.)
            issue_s(0, 0);
            issue_s(1, 0);
            if (nB == 1) mma_commit(bar + kBarQEmpty);
            // (The issuer polls for P: a suspended wait resumes some 500 cycles late,
            // which the softmax chain, bounding the kernel, would pay twice a step:
            // 1972 -> 1732 us at 32K tokens x 8 heads.)
            for (int t = 0; t < nB; ++t) {
              // tile A's burst: P_A(t) (whose arrival vouches for step t's entry, and
              // for t = 0 for the item before's O having been read)
              if (t < nA) {
                if (!(ok = mbar_wait_spin_bounded(bar + kBarPFull, (doneA + t) & 1, abort_flag, gst))) break;
                tc_fence_after_sync();
                issue_pv(0, t);
                if (t == nA - 1)
                  mma_commit(bar + kBarODone);
                else
                  issue_s(0, t + 1);
              }
              // then tile B's: P_B(t) (vouching for the entry if A skipped it)
              if (!(ok = mbar_wait_spin_bounded(bar + kBarPFull + 8, (e0 + t) & 1, abort_flag, gst))) break;
              tc_fence_after_sync();
              issue_pv(1, t);
              if (t == nB - 1)
                mma_commit(bar + kBarODone + 8);
              else
                issue_s(1, t + 1);
              if (t == nB - 2) mma_commit(bar + kBarQEmpty);
              mma_commit(bar + kBarKVEmpty + 8 * ring_slot(e0 + t));  // the entry is free
            }
            if (!ok) break;
            e0 += nB, doneA += nA;
          }
          mbar_arrive(bar + kBarItemEmpty + 8 * (n & 1));
          if (!(ok = mbar_wait_bounded(bar + kBarItem + 8 * ((n + 1) & 1), item_parity(n + 1), abort_flag, gst))) break;
          it = get_item(item_slot(n + 1));
        }
        // All tensor-core work of this CTA is complete once this commit lands.
        mma_commit(bar + kBarDrain);
        volatile int never = 0;
        mbar_wait_bounded(bar + kBarDrain, 0, &never, nullptr);
      }
    }
  } else {
    regs_inc<W::kRegsSoftmax>();
    // ------------------------- softmax: tile x (wide: half g of its keys)
    const int x = kWide ? warp >> 3 : warp >> 2, g = kWide ? (warp >> 2) & 1 : 0, w4 = warp & 3;
    const int row = w4 * 32 + lane;  // query row in the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
    const uint32_t tS = tmem + lane_base + x * BN + g * 64;
    constexpr int kOCols = D / W::kRowThreads;  // columns of O this thread writes
    const uint32_t tO = tmem + lane_base + 2 * BN + x * D + g * kOCols;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int e0 = 0, done = 0, n_live = 0;  // ring entries, this tile's steps and the items with keys before
    // The keys that this thread's row of an item sees, {first, how many}.
    auto keys_of = [&](const Item &it) -> int2 {
      const int pos = it.tile * 2 * BM + x * BM + row;
      if (!p.mod.mask.ranges) return make_int2(0, p.causal ? min(pos + 1, p.S) : p.S);
      const long long ri = (long long)(it.rb % p.B) * p.mod.mask.Sp + pos;  // (tile B may lie past Sp)
      return pos < p.mod.mask.Sp && in_range(p.status, ri, 1, p.mod.mask.rows_n) ? __ldg(p.mod.mask.ranges + ri)
                                                                                 : make_int2(0, 0);
    };
    int2 keys = keys_of(get_item(item_slot(0)));
#pragma unroll 1
    for (int n = 0;; ++n) {
      const Item it = get_item(item_slot(n));
      const int n_mine = x ? it.nB : it.nA;
      const int own_entry_from = x ? it.nA : 0;  // steps whose first burst is this tile's
      // The keys this row sees, [k_lo, k_hi).  A row that sees none (or lies past the
      // sequence) is computed as if it saw all (and more: k_lo < 0), so that it costs
      // its warp no masking, and written as O = 0, LSE = -inf.
      const int k_lo = keys.y == 0 ? -(1 << 29) : keys.x, k_hi = keys.y == 0 ? 1 << 29 : keys.x + keys.y;
      float m_used = kWide ? 0.f : -INFINITY, l = 0.f;  // the row's reference (base 2) and sum
      // wide: what the rounded P of masked steps add to that.  No reference makes a
      // row's largest P 1, so its rounding, up to 2^-8 of it, would stay in O of a
      // row that sees one key: O is divided by the sum of what V was multiplied by.
      // In other steps it does stay: where one key of many carries a row, O is off
      // by as much, as in the narrow form once a row's maximum has left its
      // reference behind.  (This costs 8K tokens x 32 heads in documents of random
      // lengths about 1024 170 -> 183 us.)
      float l_off = 0.f, lse_sum = 0.f;
      int form = 0;  // the form of tanh this warp's tiles have needed so far
      // The MMA issuer waits for P_x(t)'s arrivals alone; when that burst is the
      // step's first, they also vouch for the ring entry having landed.
      auto publish = [&](int t) -> bool {
        tmem_wait_st();
        tc_fence_before_sync();
        if (t >= own_entry_from &&
            !warp_wait(bar + kBarKVFull + 8 * ring_slot(e0 + t), ring_parity(e0 + t), abort_flag, gst))
          return false;
        mbar_arrive(bar + kBarPFull + 8 * x);
        return true;
      };
      if constexpr (kWide) {
        const dev::Poly<2> short_form(p.mod.c2);
        for (int t = 0; t < n_mine; ++t) {
          if (!warp_wait(bar + kBarSFull + 8 * x, (done + t) & 1, abort_flag, gst)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          // columns [first, first + len) are seen
          const int first = k_lo - (tile_of(it, t) * BN + 64 * g), len = k_hi - k_lo;
          const bool part = __any_sync(0xffffffffu, first > 0 || first + len < 64);
          uint32_t w[2][16];
          float tsum, toff;
          // P of the thread's 64 scores in form kForm, 16 at a time, into w (the
          // scores in TMEM stay until the form is known to do); the
          // largest square of a score.
          auto exps = [&](auto form_c, auto mask_c) -> float {
            using namespace dev;
            constexpr int kForm = decltype(form_c)::value;
            constexpr bool kMask = decltype(mask_c)::value;
            const Poly<4> long_form(p.mod.c4);
            const CapAny any(p.mod);
            f2x rs[2] = {f2_of(0.f, 0.f), f2_of(0.f, 0.f)}, in_v = rs[0];
            float bg[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t seen = 0xffffu;  // columns of the 16 that the row sees
              if constexpr (kMask) {
                seen = bits_of(first - 16 * c, first - 16 * c + len) & 0xffffu;
                if (!__any_sync(0xffffffffu, seen != 0u)) {  // nobody in the warp sees any
#pragma unroll
                  for (int e = 0; e < 8; ++e) w[c >> 1][(c & 1) * 8 + e] = 0u;
                  continue;
                }
              }
              uint32_t s[16];
              tmem_ld16(tS + c * 16, s);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(s[i]));  // no use before the wait
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                f2x v[2] = {f2_of(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])),
                            f2_of(__uint_as_float(s[2 * e + 2]), __uint_as_float(s[2 * e + 3]))};
                if constexpr (kForm == 2) {
                  // (four scores share a reciprocal, and what is unseen may be NaN.  202 ->
                  // 212 us in documents of random lengths about 1024, 8K tokens x 32 heads,
                  // all in this form; a look whether any is NaN first, or another pass if
                  // one was: 215-228.)
                  if constexpr (kMask) any.drop_unseen(v[0], v[1], seen >> (2 * e));
                  any(v[0], v[1]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  if constexpr (kForm < 2) {
                    const f2x u = f2_mul(v[h], v[h]);
                    const float2 u2 = f2_to(u);
                    bg[h] = max3(bg[h], u2.x, u2.y);
                    if constexpr (kForm == 0)
                      v[h] = f2_mul(v[h], short_form(u));
                    else
                      v[h] = f2_mul(v[h], long_form(u));
                  }
                  const float2 y = f2_to(v[h]);
                  float2 pe = make_float2(ex2(y.x), ex2(y.y));
                  if constexpr (kMask) {
                    if (!(seen & (1u << (2 * (e + h))))) pe.x = 0.f;
                    if (!(seen & (2u << (2 * (e + h))))) pe.y = 0.f;
                  }
                  rs[h] = f2_add(rs[h], f2_of(pe.x, pe.y));
                  const uint32_t rounded = pack_bf16x2(pe.x, pe.y);
                  w[c >> 1][(c & 1) * 8 + e + h] = rounded;
                  if constexpr (kMask)
                    in_v = f2_add(in_v, f2_of(__uint_as_float(rounded << 16),
                                                      __uint_as_float(rounded & 0xffff0000u)));
                }
              }
            }
            const float2 sum = f2_to(f2_add(rs[0], rs[1]));
            tsum = sum.x + sum.y;
            const float2 r2 = f2_to(in_v);
            toff = kMask ? (r2.x + r2.y) - tsum : 0.f;
            return fmaxf(bg[0], bg[1]);
          };
          using std::integral_constant;
#pragma unroll 1
          for (;;) {
            float big;
            if (part)
              big = form == 0   ? exps(integral_constant<int, 0>{}, std::true_type{})
                    : form == 1 ? exps(integral_constant<int, 1>{}, std::true_type{})
                                : exps(integral_constant<int, 2>{}, std::true_type{});
            else
              big = form == 0   ? exps(integral_constant<int, 0>{}, std::false_type{})
                    : form == 1 ? exps(integral_constant<int, 1>{}, std::false_type{})
                                : exps(integral_constant<int, 2>{}, std::false_type{});
            if (form == 2 || !__any_sync(0xffffffffu, big > (form == 0 ? p.mod.lim2 : p.mod.lim4))) break;
            form = dev::cap_form(big, p.mod);
          }
          // (half g's P lies over the first half of its own scores)
          tmem_st16(tS, w[0]);
          tmem_st16(tS + 16, w[1]);
          l += tsum;
          l_off += toff;
          if (!publish(t)) {
            ok = false;
            break;
          }
        }
        // The row's sum: both halves', added in the same order by both.
        if (n_mine > 0) {
          volatile float *red = reinterpret_cast<volatile float *>(smem + L::kRed) + x * 256 + row;
          volatile int16_t *off1 = reinterpret_cast<volatile int16_t *>(smem + L::kOff) + x * 128 + row;
          const float lo = l + l_off;
          if (ok && n_live > 0) ok = warp_wait(bar + kBarRead + 8 * x, (n_live - 1) & 1, abort_flag, gst);
          if (ok) {
            red[g * 128] = lo;
            if (g == 1) *off1 = (int16_t)(lo > 0.f ? __float2int_rn(l_off / lo * 4194304.f) : 0);  // (at most 2^-8)
            mbar_arrive(bar + kBarSum + 8 * x);
            ok = warp_wait(bar + kBarSum + 8 * x, n_live & 1, abort_flag, gst);
            // half 0 writes the LSE, from the unrounded sum: its own, and half 1's
            const float lo1 = red[128];
            if (g == 0) lse_sum = l + fmaf(lo1, (float)*off1 * (-1.0f / 4194304.f), lo1);
            l = red[0] + lo1;
            mbar_arrive(bar + kBarRead + 8 * x);
          }
        }
      } else {
        // the scale of what exps reads: raw scores, or (capped, biased) base-2 logits
        const float xs = kCap || kBias ? 1.0f : sl2;
        float slope2 = 0.f;
        if constexpr (kBias) slope2 = dev::slope_at(p.mod, (it.rb / p.B) * p.hp + it.j, p.Pu * p.hp, p.status);
        for (int t = 0; t < n_mine; ++t) {
          if (!warp_wait(bar + kBarSFull + 8 * x, (done + t) & 1, abort_flag, gst)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) reg_fence(s[c]);
          const int kv0 = tile_of(it, t) * BN, pos = it.tile * 2 * BM + x * BM + row;
          const int c0 = k_lo - kv0, c1 = k_hi - kv0;  // columns [c0, c1) are seen
          const bool part = __any_sync(0xffffffffu, c0 > 0 || c1 < BN);
          dev::LinearBias lb{true, 0.f, 0.f};
          if constexpr (kBias) lb = dev::linear_bias<BN>(slope2, kv0 - pos);
          // `raw`: the exponentials read the scores as they are (nothing masked,
          // every row's reference set, the bias linear); else these become base-2
          // logits in place first, masked ones -inf.
          bool raw = (kCap || kBias) && !part && lb.ok && !__any_sync(0xffffffffu, m_used == -INFINITY);
          auto make_logits = [&]() { dev::logits<kMod>(s, p.mod, sl2, slope2, kv0 - pos, part, c0, c1); };
          if (!raw) {
            make_logits();
            if (part) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t seen = bits_of(c0 - 32 * c, c1 - 32 * c);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(seen & (1u << e))) s[c][e] = __float_as_uint(-INFINITY);
              }
            }
          }
          // Row maximum: eight independent chains of three-input maxima over 16 columns each.
          auto row_max = [&]() -> float {
            float mx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t *r = &s[i >> 1][(i & 1) * 16];
              float m = max3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]));
#pragma unroll
              for (int e = 3; e < 15; e += 2) m = max3(m, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
              mx[i] = fmaxf(m, __uint_as_float(r[15]));
            }
            return fmaxf(max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])), -INFINITY);
          };
          // P = exp2(xs * s - m) into the first 64 columns of S (bf16, two keys
          // per column); returns the row's sum of P.
          auto exps = [&](float m) -> float {
            const float2 sl22 = make_float2(xs, xs), nb2 = make_float2(-m, -m);
            float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 sp = make_float2(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1]));
                const float2 a = kCap || kBias ? add2(sp, nb2) : fma2(sp, sl22, nb2);
                const float2 pe = make_float2(ex2(a.x), ex2(a.y));
                rs[e & 1] = add2(rs[e & 1], pe);
                w[e] = pack_bf16x2(pe.x, pe.y);
              }
              tmem_st16(tS + c * 16, w);
            }
            return (rs[0].x + rs[1].x) + (rs[0].y + rs[1].y);
          };
          // The same from raw scores: tanh in form kForm, the bias and the offset
          // in one multiply-add; `big` is the largest square.
          auto exps_raw = [&](auto form_c, float m, float &big) -> float {
            using namespace dev;
            constexpr int kForm = decltype(form_c)::value;
            f2x rs[2] = {f2_of(0.f, 0.f), f2_of(0.f, 0.f)};
            [[maybe_unused]] const float base = lb.base - m;
            const f2x minus_m = f2_const(-m), scale2 = f2_const(sl2);
            const Poly<2> short_form(p.mod.c2);
            const Poly<4> long_form(p.mod.c4);
            const CapAny any(p.mod);
            const BiasSteps steps(lb);
            float bg[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const uint32_t *r = &s[c][2 * e];
                f2x v[2] = {f2_of(__uint_as_float(r[0]), __uint_as_float(r[1])),
                            f2_of(__uint_as_float(r[2]), __uint_as_float(r[3]))};
                if constexpr (kCap && kForm == 2) any(v[0], v[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  f2x add = minus_m;
                  if constexpr (kBias) {
                    const float b16 = fmaf((float)(32 * c + (e & 8) * 2), lb.slope2, base);
                    add = f2_add(steps.d[(e & 7) + h], f2_of(b16, b16));
                  }
                  f2x y;
                  if constexpr (!kCap)
                    y = f2_fma(v[h], scale2, add);
                  else if constexpr (kForm < 2) {
                    const f2x u = f2_mul(v[h], v[h]);
                    const float2 u2 = f2_to(u);
                    bg[h] = max3(bg[h], u2.x, u2.y);
                    if constexpr (kForm == 0)
                      y = f2_fma(v[h], short_form(u), add);
                    else
                      y = f2_fma(v[h], long_form(u), add);
                  } else {
                    y = f2_add(v[h], add);
                  }
                  const float2 y2 = f2_to(y);
                  const float2 pe = make_float2(ex2(y2.x), ex2(y2.y));
                  rs[h] = f2_add(rs[h], f2_of(pe.x, pe.y));
                  w[e + h] = pack_bf16x2(pe.x, pe.y);
                }
              }
              tmem_st16(tS + c * 16, w);
            }
            big = fmaxf(bg[0], bg[1]);
            const float2 sum = f2_to(f2_add(rs[0], rs[1]));
            return sum.x + sum.y;
          };
          // The reference only guards against overflow (the exponentials' relative
          // precision does not depend on it): it is set from the row maximum on
          // the first tile in which the row sees a key and afterwards moved only
          // when a tile's row sum of P passes 2^16 (some score more than 9 above
          // it); that tile's P is then formed again and O and l are rescaled.
          float tsum = 0.f;
          if constexpr (kCap || kBias) {
#pragma unroll 1
            while (raw) {
              float big = 0.f;
              if constexpr (kCap) {
                tsum = form == 0   ? exps_raw(std::integral_constant<int, 0>{}, m_used, big)
                       : form == 1 ? exps_raw(std::integral_constant<int, 1>{}, m_used, big)
                                   : exps_raw(std::integral_constant<int, 2>{}, m_used, big);
                const int need_form = form == 2 ? 2 : dev::cap_form(big, p.mod);
                if (need_form > form) {
                  form = need_form;
                  continue;
                }
              } else {
                tsum = exps_raw(std::integral_constant<int, 0>{}, m_used, big);
              }
              if (!__any_sync(0xffffffffu, !(tsum <= 65536.0f))) break;  // (leaves with inf and NaN too)
              make_logits();
              raw = false;
            }
          }
          bool need = m_used == -INFINITY || (!raw && tsum != 0.f);  // (a raw pass that overflowed: all rows look)
#pragma unroll 1
          for (int pass = raw ? 2 : 0; pass < 2; ++pass) {
            if (__any_sync(0xffffffffu, need)) {
              // (the commit of S_X(t) that was waited for also covers PV_X(t-1):
              // no MMA touches O_X until P_X(t) is published)
              const float ms = need ? fmaxf(row_max() * xs, m_used) : m_used;
              const float alpha = m_used == -INFINITY || ms == m_used ? 1.f : ex2(m_used - ms);
              if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1  // (unrolled, it spills)
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t r[32];
                  tmem_ld32(tO + c * 32, r);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 32; e += 2) {
                    const float2 v = mul2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])),
                                          make_float2(alpha, alpha));
                    r[e] = __float_as_uint(v.x);
                    r[e + 1] = __float_as_uint(v.y);
                  }
                  tmem_st32(tO + c * 32, r);
                }
                tmem_wait_st();
                l *= alpha;
              }
              m_used = ms;
            }
            tsum = exps(m_used == -INFINITY ? 0.f : m_used);  // (-inf: nothing seen yet, P = 0)
            if (pass == 1) break;
            need = !(tsum <= 65536.0f);  // also true for inf
            if (!__any_sync(0xffffffffu, need)) break;
          }
          l += tsum;
          if (!publish(t)) {
            ok = false;
            break;
          }
        }
      }
      // The row's keys in the next item come on their way through the epilogue.
      if (ok) ok = warp_wait(bar + kBarItem + 8 * ((n + 1) & 1), item_parity(n + 1), abort_flag, gst);
      bool more = false;
      if (ok) {
        const Item next = get_item(item_slot(n + 1));
        more = next.tile >= 0;
        if (more) keys = keys_of(next);
      }
      const Item cur = get_item(item_slot(n));
      const int qpos = cur.tile * 2 * BM + x * BM + row;
      const bool dead = k_lo < 0;
      // --------------------------------------------------------------- epilogue
      if (ok && n_mine > 0) ok = warp_wait(bar + kBarODone + 8 * x, n_live & 1, abort_flag, gst);
      if (ok) {
        tc_fence_after_sync();
        const float inv = 1.0f / l;
        const size_t hr = (size_t)(qpos / p.Cs) * p.Pu * p.B + cur.rb;  // head-layout rank * B + b
        const size_t ooff = ((hr * p.Cs + qpos % p.Cs) * p.hp + cur.j) * D + g * kOCols;
        const bool store = qpos < p.S && in_range(p.status, (long long)ooff, kOCols, p.o_n);
#pragma unroll
        for (int c = 0; c < kOCols / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(tO + c * 32, r);  // (of an item without keys: what it holds is not used)
          tmem_wait_ld();
          if (store) {
            __nv_bfloat16 *dst = p.o + ooff + c * 32;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e] = dead ? 0u
                            : pack_bf16x2(__uint_as_float(r[16 * v + 2 * e]) * inv,
                                          __uint_as_float(r[16 * v + 2 * e + 1]) * inv);
              if (p.o_by32) {
                st_global_32(dst + 16 * v, w);
              } else {
                reinterpret_cast<uint4 *>(dst + 16 * v)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4 *>(dst + 16 * v)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
        if (g == 0 && qpos < p.S) {
          const size_t li = (hr * p.hp + cur.j) * p.Cs + qpos % p.Cs;
          if (in_range(p.status, (long long)li, 1, p.lse_n))
            p.lse[li] = dead ? -INFINITY : (m_used + log2f(kWide ? lse_sum : l)) * 0.69314718055994530942f;
        }
      }
      if (!ok || !more) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + kBarItemEmpty + 8 * (n & 1));
      e0 += cur.nB, done += n_mine, n_live += cur.nB > 0 ? 1 : 0;
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, (uint32_t)ULYSSES_STATUS_FWD_TIMEOUT);
}

template <int D, int kMod, bool kWide = false>
cudaError_t launch_as(const FwdParams &fp, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                      unsigned blocks, cudaStream_t st) {
  const auto kernel = attn_fwd_mod_tc_kernel<D, kMod, kWide>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, Roles<kWide>::kThreads, Layout<D>::kAlloc, st>>>(mq, mk, mv, fp);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const ulysses_problem &p, const TmaEncoder &enc, const void *q, const void *k, const void *v,
                     void *o, float *lse, uint32_t *status, const ulysses_score_mod &m, cudaStream_t st) {
  const int Pu = group_ranks(p), Cs = chunk_len(p);
  const int hp = p.n_head / Pu, kvp = kv_per_rank(p), PB = p.P * p.B;
  CUtensorMap mq, mk, mv;  // [P*B][Cs][hp|kvp][D]
  if (!make_act_map(enc, &mq, q, D, hp, Cs, PB, 128) || !make_act_map(enc, &mk, k, D, kvp, Cs, PB, 128) ||
      !make_act_map(enc, &mv, v, D, kvp, Cs, PB, 128))
    return cudaErrorInvalidValue;
  FwdParams fp;
  fp.B = p.B;
  fp.S = p.S;
  fp.hp = hp;
  fp.kvp = kvp;
  fp.group = hp / kvp;
  fp.causal = p.causal;
  fp.n_pairs = (p.S + 2 * BM - 1) / (2 * BM);
  fp.Pu = Pu;
  fp.Cs = Cs;
  const float scale = p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf((float)D);
  fp.scale_log2 = scale * 1.4426950408889634f;
  const int units = Pu * p.B * hp;  // (group member, batch, local head): one full-sequence head each
  fp.head_group = l2_head_group((size_t)4 * p.S * D / fp.group, units, (long long)fp.n_pairs * units, (size_t)32 << 20);
  fp.o = static_cast<__nv_bfloat16 *>(o);
  fp.o_by32 = (reinterpret_cast<uintptr_t>(o) & 31) == 0;
  fp.lse = lse;
  fp.o_n = (long long)p.B * p.S * p.n_head * D;
  fp.lse_n = (long long)p.B * p.n_head * p.S;
  fp.status = status;
  fp.mod = score_mod(p, m);
  const long long blocks = (long long)fp.n_pairs * units;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const unsigned nb = (unsigned)blocks;
  switch (score_mod_flags(m)) {
    case kModOn: return launch_as<D, kModOn>(fp, mq, mk, mv, nb, st);
    case kModOn | kModCap:
      if (fp.mod.cap_out <= 80.f) return launch_as<D, kModOn | kModCap, true>(fp, mq, mk, mv, nb, st);
      return launch_as<D, kModOn | kModCap>(fp, mq, mk, mv, nb, st);
    case kModOn | kModBias: return launch_as<D, kModOn | kModBias>(fp, mq, mk, mv, nb, st);
    case kModOn | kModCap | kModBias: return launch_as<D, kModOn | kModCap | kModBias>(fp, mq, mk, mv, nb, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_attn_fwd_mod_tc(const ulysses_problem &p, const TmaEncoder &enc, const void *q, const void *k,
                                   const void *v, void *o, float *lse, uint32_t *status,
                                   const ulysses_score_mod &mod, cudaStream_t st) {
  if (p.head_dim == 128) return launch_d<128>(p, enc, q, k, v, o, lse, status, mod, st);
  if (p.head_dim == 64) return launch_d<64>(p, enc, q, k, v, o, lse, status, mod, st);
  return cudaErrorInvalidValue;
}

}  // namespace ulysses
