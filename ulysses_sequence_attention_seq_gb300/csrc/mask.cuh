// mask.cuh -- the mask plan: which keys every query row sees, and which
// 128 x 128 tiles of the scores hold anything.
//
// Every mask the attention takes (causal, documents, prefixes, a window,
// padding) leaves a row one interval of keys, [lo, lo + len): two ints a row
// say all of it.  The plan also holds, per 128-row query tile, the hull of its
// rows' intervals and the keys that all of them see, and, per 128-key tile,
// the list of query tiles whose hull meets it.  Kernels then skip tile pairs
// that are empty and mask only those that are not full.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "check.cuh"
#include "internal.h"

namespace ulysses {
namespace dev {

struct MaskView {
  // [B][Sp] {lo, len}, Sp = S rounded up to 128; rows past S, and rows that
  // see nothing, have len 0.  Null: no plan (the problem's causal flag alone).
  const int2 *ranges;
  // [B][Sp] the queries that see a key, {first, count}: an interval too where
  // both ends of the rows' intervals rise along the batch row (documents,
  // windows, a prefix length that is the same for a whole document).  Count -1
  // where they do not.
  const int2 *keys;
  // [B][n_t] per query tile: x, y = hull [x, y) of its rows' intervals (x >= y:
  // all empty); z, w = keys [z, w) that all of its rows see but those that see
  // nothing (none with rows past S).
  const int4 *tiles;
  const int *col_n;      // [B][n_t] query tiles that see a key tile ...
  const uint16_t *cols;  // [B][n_t][n_t] ... in rising order: 2 * tile + (nothing of the pair needs masking)
  const int2 *order;     // [B][n_t] {key tile, its query tiles}, those with most first
  const uint64_t *head;  // {key}
  uint64_t key;          // B, S and the causal flag themselves: no two problems share one
  int Sp, n_t;
  long long rows_n;      // B * Sp
};

// The plan's key: not m.key where it was built for another problem.  (Read it
// first and look at it once the block's other loads are on their way.)
__device__ __forceinline__ uint64_t mask_key_of(const MaskView &m) { return m.ranges ? __ldg(m.head) : m.key; }
__device__ __forceinline__ bool mask_matches(const MaskView &m) { return mask_key_of(m) == m.key; }

__device__ __forceinline__ bool row_empty(const MaskView &m, int b, int pos, uint32_t *status) {
  if (!m.ranges) return false;
  const long long i = (long long)b * m.Sp + pos;
  return !in_range(status, i, 1, m.rows_n) || __ldg(&m.ranges[i].y) == 0;
}

// Entries of the plan, range-checked in a checked build: query tile i's
// {hull, common keys} and the i-th key tile in order (both of B * n_t), and entry
// i of the lists (B * n_t * n_t).
__device__ __forceinline__ int4 tile_at(const MaskView &m, long long i, uint32_t *status) {
  return in_range(status, i, 1, m.rows_n / 128) ? __ldg(m.tiles + i) : make_int4(INT_MAX, 0, INT_MAX, 0);
}
__device__ __forceinline__ int2 order_at(const MaskView &m, long long i, uint32_t *status) {
  return in_range(status, i, 1, m.rows_n / 128) ? __ldg(m.order + i) : make_int2(0, 0);
}
__device__ __forceinline__ int col_at(const MaskView &m, const uint16_t *list, int i, uint32_t *status) {
  return in_range(status, list - m.cols + i, 1, m.rows_n / 128 * m.n_t) ? __ldg(list + i) : 0;
}

}  // namespace dev

// Byte offsets inside a mask plan (256-aligned; the first 256 bytes: the key).
// `edges` is used while the plan is built and then holds the order.
struct MaskLayout {
  size_t ranges = 0, keys = 0, tiles = 0, ends = 0, edges = 0, col_n = 0, cols = 0, total = 0;
};
MaskLayout mask_layout(const ulysses_problem &p);
dev::MaskView mask_view(const ulysses_problem &p, const void *mask);

}  // namespace ulysses
