// mask.cu -- builds the mask plan of mask.cuh from document ids, prefix
// lengths and a window.
//
// A document is a run of equal consecutive ids.  Token i of a document [a, e)
// sees, without the causal flag, [a, e); with it, [a, max(i + 1, min(e, a +
// prefix_i))); a window w cuts that to (i - w, i + w); a token with a negative
// id sees nothing, and no other token sees it, since no other run holds it.
//
// Latency is all there is (a few hundred KB at most), so up to 8192 tokens one
// launch does it all.  Above them one pass finds where runs begin in every
// 128-token tile, a second gives each token its run (a scan inside the tile, the
// neighbours' edges for what lies outside) and each tile its hull, a third lists
// the query tiles of every key tile and, where the intervals' ends rise, looks up
// every key's queries, and a fourth orders the key tiles by the length of their
// lists.
#include <limits.h>
#include <string.h>

#include "mask.cuh"

namespace ulysses {

namespace {

constexpr int kTile = 128;

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct BuildParams {
  const int *doc, *prefix;  // [B][S] or null
  int S, Sp, n_t, causal, window;
  int2 *ranges, *keys;
  int4 *tiles;
  int4 *ends;   // [B][n_t] interval of the tile's first and of its last row, {lo, hi, lo, hi} (x -1: its ends fall)
  int2 *order;
  int2 *edges;  // [B][n_t] last and first position of the tile where a run begins (-1, INT_MAX: none)
  int *col_n;
  uint16_t *cols;
  uint64_t *head;
  uint64_t key;
};

__device__ __forceinline__ bool run_begins(const int *doc, int i) { return i == 0 || doc[i] != doc[i - 1]; }

// Over the 128 threads of a block: the largest of `a` and the smallest of `b`.
__device__ __forceinline__ void block_max_min(int &a, int &b, int2 *sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    b = min(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_int2(a, b);
  __syncthreads();
  a = max(max(sh[0].x, sh[1].x), max(sh[2].x, sh[3].x));
  b = min(min(sh[0].y, sh[1].y), min(sh[2].y, sh[3].y));
}

// What token i of the run [start, end) sees; lo = hi (its run's start, so that
// documents and padding in turn still rise; 0 past S) where that is nothing.
struct Interval {
  int lo, hi;
};
__device__ __forceinline__ Interval interval_of(const BuildParams &p, int b, int i, int start, int end, bool live,
                                                bool pad) {
  int lo = start, hi = end;
  if (live && p.causal) {
    int see = i + 1;
    if (p.prefix) {
      const int pre = min(max(p.prefix[(long long)b * p.S + i], 0), p.S);
      see = max(see, min(end, start + pre));
    }
    hi = see;
  }
  if (p.window > 0) {
    lo = max(lo, i - p.window + 1);
    hi = (int)min((long long)hi, (long long)i + p.window);
  }
  if (!live) return {0, 0};
  if (pad || hi <= lo) return {start, start};
  return {lo, hi};
}
// A row's share of its tile's entry: x, w taken as minima, y, z as maxima.
// Rows that see nothing do not count for the common keys (they need no masking:
// their P is 0, or nobody reads it), rows past S leave none.
__device__ __forceinline__ int4 tile_share(const Interval &v, bool live) {
  const bool empty = v.lo >= v.hi;
  return make_int4(empty ? INT_MAX : v.lo, empty ? 0 : v.hi, !live ? INT_MAX : empty ? 0 : v.lo,
                   !live ? 0 : empty ? INT_MAX : v.hi);
}
// Whether a query tile's hull meets the key tile at k0, and needs no masking there.
__device__ __forceinline__ bool tile_sees(const int4 &t, int k0) { return t.x < k0 + kTile && t.y > k0 && t.x < t.y; }
__device__ __forceinline__ int tile_whole(const int4 &t, int k0) { return t.z <= k0 && t.w >= k0 + kTile ? 1 : 0; }

__global__ void __launch_bounds__(kTile) mask_edges_kernel(const BuildParams p) {
  __shared__ int2 sh[4];
  const int m = blockIdx.x, i = m * kTile + threadIdx.x;
  const int *doc = p.doc + (long long)blockIdx.y * p.S;
  const bool edge = i < p.S && run_begins(doc, i);
  int last = edge ? i : -1, first = edge ? i : INT_MAX;
  block_max_min(last, first, sh);
  if (threadIdx.x == 0) p.edges[(long long)blockIdx.y * p.n_t + m] = make_int2(last, first);
}

__global__ void __launch_bounds__(kTile) mask_ranges_kernel(const BuildParams p) {
  __shared__ int2 sh[4], sh2[4], rows[kTile];
  const int m = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = m * kTile + threadIdx.x;
  const bool live = i < p.S;
  int start = 0, end = p.S;
  bool pad = false;
  if (p.doc) {
    const int *doc = p.doc + (long long)b * p.S;
    const int2 *ed = p.edges + (long long)b * p.n_t;
    int before = -1, after = INT_MAX;  // the nearest edges outside this tile
    for (int t = threadIdx.x; t < p.n_t; t += kTile) {
      if (t < m) before = max(before, ed[t].x);
      if (t > m) after = min(after, ed[t].y);
    }
    block_max_min(before, after, sh);
    const bool edge = live && run_begins(doc, i);
    // the last edge at or before i, the first one after i, within the warp
    const uint32_t bits = __ballot_sync(0xffffffffu, edge);
    const int w0 = i - lane;
    const uint32_t le = bits & (0xffffffffu >> (31 - lane)), gt = lane == 31 ? 0u : bits & (0xffffffffu << (lane + 1));
    if (lane == 0) sh2[warp] = make_int2(bits ? w0 + 31 - __clz(bits) : -1, bits ? w0 + __ffs(bits) - 1 : INT_MAX);
    __syncthreads();
    start = le ? w0 + 31 - __clz(le) : -1;
    end = gt ? w0 + __ffs(gt) - 1 : INT_MAX;
    for (int w = 0; w < 4; ++w) {
      if (w < warp) start = max(start, sh2[w].x);
      if (w > warp) end = min(end, sh2[w].y);
    }
    start = max(start, before);  // position 0 is an edge: never -1 for a live row
    end = min(min(end, after), p.S);
    pad = live && doc[i] < 0;
  }
  const Interval v = interval_of(p, b, i, start, end, live, pad);
  p.ranges[(long long)b * p.Sp + i] = make_int2(v.lo, v.hi - v.lo);
  rows[threadIdx.x] = make_int2(v.lo, v.hi);
  int4 t = tile_share(v, live);
  block_max_min(t.y, t.x, sh);
  block_max_min(t.z, t.w, sh);
  const int n_rows = min(kTile, p.S - m * kTile);
  const bool falls = (int)threadIdx.x + 1 < n_rows &&
                     (rows[threadIdx.x + 1].x < v.lo || rows[threadIdx.x + 1].y < v.hi);
  const bool any_falls = __syncthreads_or(falls);
  if (threadIdx.x == 0) {
    p.tiles[(long long)b * p.n_t + m] = t;
    p.ends[(long long)b * p.n_t + m] =
        make_int4(any_falls ? -1 : rows[0].x, rows[0].y, rows[n_rows - 1].x, rows[n_rows - 1].y);
    if (m == 0 && b == 0) p.head[0] = p.key;
  }
}

// The queries [first, first + count) among [a, e) whose intervals, both of whose
// ends rise, hold `key`: the first that ends behind it, and the first that begins
// behind it.  row(i) is query i's {lo, hi}; both searches at once, three probes
// each a step, in flight together.
template <typename F>
__device__ __forceinline__ int2 queries_of(int key, int a, int e, F row) {
  int a0 = a, e0 = e, a1 = a, e1 = e;
  while (a0 < e0 || a1 < e1) {
    const int q0 = (e0 - a0) / 4, q1 = (e1 - a1) / 4;
    bool t0[3], t1[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {  // (a search that has ended reads what it may, and keeps its place)
      t0[k] = row(min(a0 + (k + 1) * q0, e - 1)).y > key;
      t1[k] = row(min(a1 + (k + 1) * q1, e - 1)).x > key;
    }
    auto narrow = [](int &lo, int &hi, int q, const bool (&t)[3]) {
      if (lo >= hi) return;
      const int m1 = lo + q, m2 = lo + 2 * q, m3 = lo + 3 * q;
      if (t[0]) {
        hi = m1;
      } else if (t[1]) {
        lo = m1 + 1, hi = m2;
      } else if (t[2]) {
        lo = m2 + 1, hi = m3;
      } else {
        lo = m3 + 1;
      }
    };
    narrow(a0, e0, q0, t0);
    narrow(a1, e1, q1, t1);
  }
  return make_int2(a0, a1 - a0);
}

// One block per key tile: its query tiles in rising order, and its keys'
// queries.
__global__ void __launch_bounds__(kTile) mask_lists_kernel(const BuildParams p) {
  __shared__ int count[4];
  const int n = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k0 = n * kTile;
  const int4 *tiles = p.tiles + (long long)b * p.n_t;
  const int4 *ends = p.ends + (long long)b * p.n_t;
  uint16_t *out = p.cols + ((long long)b * p.n_t + n) * p.n_t;
  int done = 0, m_lo = INT_MAX, m_hi = -1;  // the first and last query tile this thread lists
  bool falls = false;
  for (int m0 = 0; m0 < p.n_t; m0 += kTile) {
    const int m = m0 + threadIdx.x;
    const int4 t = m < p.n_t ? tiles[m] : make_int4(INT_MAX, 0, INT_MAX, 0);
    const bool on = tile_sees(t, k0);
    if (on) m_lo = min(m_lo, m), m_hi = m;
    if (m < p.n_t) {
      const int4 e = ends[m];
      falls |= e.x < 0;
      if (m + 1 < p.n_t) {
        const int4 next = ends[m + 1];
        falls |= next.x < e.z || next.y < e.w;  // (next.x -1 is seen by its own thread)
      }
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, on);
    __syncthreads();  // the previous chunk's counts have been read
    if (lane == 0) count[warp] = __popc(bits);
    __syncthreads();
    int at = done + __popc(bits & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) at += count[w];
    if (on) out[at] = (uint16_t)(2 * m + tile_whole(t, k0));
    done += count[0] + count[1] + count[2] + count[3];
  }
  if (threadIdx.x == 0) p.col_n[(long long)b * p.n_t + n] = done;
  __shared__ int2 sh[4];
  block_max_min(m_hi, m_lo, sh);
  const bool any_falls = __syncthreads_or(falls);
  const int key = k0 + threadIdx.x;
  int2 q = make_int2(0, any_falls ? -1 : 0);
  if (!any_falls && m_hi >= 0 && key < p.S) {
    const int2 *rg = p.ranges + (long long)b * p.Sp;
    const int a = m_lo * kTile, e = min(m_hi * kTile + kTile, p.S);
    q = queries_of(key, a, e, [&](int i) {
      const int2 r = rg[i];
      return make_int2(r.x, r.x + r.y);
    });
  }
  p.keys[(long long)b * p.Sp + key] = q;
}

// Up to kSmall tokens: everything in one launch, one block a batch row, a thread
// a token, the rows' intervals in shared memory: 97 tokens x 2 3.4 us, 1024 5.0
// us, where the four launches take 10.  (Four tokens a thread instead of more
// blocks: 2060 tokens 12 us.)
constexpr int kSmall = 1024;

__global__ void __launch_bounds__(kSmall) mask_small_kernel(const BuildParams p) {
  __shared__ uint32_t edge_bits[32];
  __shared__ int2 rows[kSmall];
  __shared__ int4 warp_tile[32], tile[kSmall / kTile];
  const int i = threadIdx.x, b = blockIdx.x, lane = i & 31, warp = i >> 5;
  const bool live = i < p.S;
  int start = 0, end = p.S;
  bool pad = false;
  if (p.doc) {
    const int *doc = p.doc + (long long)b * p.S;
    const uint32_t bits = __ballot_sync(0xffffffffu, live && run_begins(doc, i));
    if (lane == 0) edge_bits[warp] = bits;
    __syncthreads();
    // lane l: the last and the first edge of warp l's tokens
    const uint32_t theirs = edge_bits[lane];
    int before = lane < warp && theirs ? 32 * lane + 31 - __clz(theirs) : -1;
    int after = lane > warp && theirs ? 32 * lane + __ffs(theirs) - 1 : INT_MAX;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before = max(before, __shfl_xor_sync(0xffffffffu, before, o));
      after = min(after, __shfl_xor_sync(0xffffffffu, after, o));
    }
    const uint32_t le = bits & (0xffffffffu >> (31 - lane)), gt = lane == 31 ? 0u : bits & (0xffffffffu << (lane + 1));
    start = le ? 32 * warp + 31 - __clz(le) : before;
    end = min(gt ? 32 * warp + __ffs(gt) - 1 : after, p.S);
    pad = live && doc[i] < 0;
  }
  const Interval v = interval_of(p, b, i, start, end, live, pad);
  const bool on = i < p.Sp;
  if (on) p.ranges[(long long)b * p.Sp + i] = make_int2(v.lo, v.hi - v.lo);
  rows[i] = make_int2(v.lo, v.hi);
  int4 t = tile_share(v, live);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t.x = min(t.x, __shfl_xor_sync(0xffffffffu, t.x, o));
    t.y = max(t.y, __shfl_xor_sync(0xffffffffu, t.y, o));
    t.z = max(t.z, __shfl_xor_sync(0xffffffffu, t.z, o));
    t.w = min(t.w, __shfl_xor_sync(0xffffffffu, t.w, o));
  }
  if (lane == 0) warp_tile[warp] = t;
  __syncthreads();
  const bool falls = i + 1 < p.S && (rows[i + 1].x < v.lo || rows[i + 1].y < v.hi);
  const bool any_falls = __syncthreads_or(falls);
  if (i < p.n_t) {
    const int4 a = warp_tile[4 * i], c = warp_tile[4 * i + 1], d = warp_tile[4 * i + 2], e = warp_tile[4 * i + 3];
    t = make_int4(min(min(a.x, c.x), min(d.x, e.x)), max(max(a.y, c.y), max(d.y, e.y)),
                  max(max(a.z, c.z), max(d.z, e.z)), min(min(a.w, c.w), min(d.w, e.w)));
    tile[i] = t;
    p.tiles[(long long)b * p.n_t + i] = t;
  }
  if (i == 0 && b == 0) p.head[0] = p.key;
  __syncthreads();
  if (i < p.n_t) {  // key tile i's query tiles
    uint16_t *out = p.cols + ((long long)b * p.n_t + i) * p.n_t;
    int n = 0;
    for (int m = 0; m < p.n_t; ++m)
      if (tile_sees(tile[m], i * kTile)) out[n++] = (uint16_t)(2 * m + tile_whole(tile[m], i * kTile));
    p.col_n[(long long)b * p.n_t + i] = n;
    p.order[(long long)b * p.n_t + i] = make_int2(i, n);  // (too few to matter)
  }
  if (on) {
    int2 q = make_int2(0, any_falls ? -1 : 0);
    if (!any_falls && live) {
      q = queries_of(i, 0, p.S, [&](int r) { return rows[r]; });
    }
    p.keys[(long long)b * p.Sp + i] = q;
  }
}

// A batch row's key tiles by falling number of their query tiles: the order in
// which dK/dV takes them, whose items differ most in length and are fewest
// (packed documents, 8K tokens x 8 kv-heads: 688 -> 633 us of backward).
// Each tile counts those before it; above kOrder tiles, where one row's items
// fill the GPU many times over, they stay in their own order.
constexpr int kOrder = 1024;

__global__ void __launch_bounds__(256) mask_order_kernel(const BuildParams p) {
  __shared__ int count[kOrder];
  const int *n = p.col_n + (long long)blockIdx.x * p.n_t;
  int2 *order = p.order + (long long)blockIdx.x * p.n_t;
  if (p.n_t > kOrder) {
    for (int i = threadIdx.x; i < p.n_t; i += 256) order[i] = make_int2(i, n[i]);
    return;
  }
  for (int i = threadIdx.x; i < p.n_t; i += 256) count[i] = n[i];
  __syncthreads();
  for (int i = threadIdx.x; i < p.n_t; i += 256) {
    const int c = count[i];
    int rank = 0;
    for (int j = 0; j < p.n_t; ++j) rank += count[j] > c || (count[j] == c && j < i) ? 1 : 0;
    order[rank] = make_int2(i, c);
  }
}

// Up to kMiddle tokens: a cluster of blocks a batch row, 1024 tokens a block, and
// barriers of the cluster where the kernels above end; what they hand on goes
// through the plan itself.  2060 tokens x 2 9 us, 8192 11 us; the four launches
// above take as long one behind the other, but 21 us called one by one.
constexpr int kMiddle = 8 * kSmall;

// (Every thread of the block calls it, but after branches that differ from lane to
// lane: so not the .aligned forms, which want a warp's lanes together.)
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__global__ void __launch_bounds__(kSmall) mask_cluster_kernel(const BuildParams p) {
  __shared__ uint32_t edge_bits[32];
  __shared__ int2 rows[kSmall];
  __shared__ int4 warp_tile[32];
  __shared__ int2 listed[kSmall / kTile];  // first and last query tile of each of the block's key tiles
  const int c = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = c * kSmall, i = first + threadIdx.x, blocks = (p.S + kSmall - 1) / kSmall;  // (with tokens)
  const long long at = (long long)b * p.n_t;
  const bool live = i < p.S;
  int start = 0, end = p.S;
  bool pad = false;
  if (p.doc) {
    const int *doc = p.doc + (long long)b * p.S;
    const uint32_t bits = __ballot_sync(0xffffffffu, live && run_begins(doc, i));
    if (lane == 0) edge_bits[warp] = bits;
    __syncthreads();
    const uint32_t theirs = edge_bits[lane];  // of the block's warp `lane`
    const int their_last = theirs ? first + 32 * lane + 31 - __clz(theirs) : -1;
    const int their_first = theirs ? first + 32 * lane + __ffs(theirs) - 1 : INT_MAX;
    if (warp == 0) {
      const int last = __reduce_max_sync(0xffffffffu, their_last), fst = __reduce_min_sync(0xffffffffu, their_first);
      if (lane == 0) p.edges[at + c] = make_int2(last, fst);
    }
    cluster_barrier();
    int before = lane < warp ? their_last : -1, after = lane > warp ? their_first : INT_MAX;
    if (lane < blocks && lane != c) {
      const int2 e = __ldcg(p.edges + at + lane);
      if (lane < c) before = max(before, e.x);
      if (lane > c) after = min(after, e.y);
    }
    before = __reduce_max_sync(0xffffffffu, before);
    after = __reduce_min_sync(0xffffffffu, after);
    const uint32_t le = bits & (0xffffffffu >> (31 - lane)), gt = lane == 31 ? 0u : bits & (0xffffffffu << (lane + 1));
    start = le ? first + 32 * warp + 31 - __clz(le) : before;
    end = min(gt ? first + 32 * warp + __ffs(gt) - 1 : after, p.S);
    pad = live && doc[i] < 0;
  }
  const Interval v = interval_of(p, b, i, start, end, live, pad);
  const bool on = i < p.Sp;
  if (on) p.ranges[(long long)b * p.Sp + i] = make_int2(v.lo, v.hi - v.lo);
  rows[threadIdx.x] = make_int2(v.lo, v.hi);
  int4 t = tile_share(v, live);
  t.x = __reduce_min_sync(0xffffffffu, t.x);
  t.y = __reduce_max_sync(0xffffffffu, t.y);
  t.z = __reduce_max_sync(0xffffffffu, t.z);
  t.w = __reduce_min_sync(0xffffffffu, t.w);
  if (lane == 0) warp_tile[warp] = t;
  __syncthreads();
  const int n_rows = min(kSmall, p.S - first);
  const bool falls =
      (int)threadIdx.x + 1 < n_rows && (rows[threadIdx.x + 1].x < v.lo || rows[threadIdx.x + 1].y < v.hi);
  const bool any = __syncthreads_or(falls);
  const int mine = threadIdx.x < kSmall / kTile ? c * (kSmall / kTile) + (int)threadIdx.x : p.n_t;
  if (mine < p.n_t) {
    const int4 *w = warp_tile + 4 * threadIdx.x;
    p.tiles[at + mine] = make_int4(min(min(w[0].x, w[1].x), min(w[2].x, w[3].x)),
                                   max(max(w[0].y, w[1].y), max(w[2].y, w[3].y)),
                                   max(max(w[0].z, w[1].z), max(w[2].z, w[3].z)),
                                   min(min(w[0].w, w[1].w), min(w[2].w, w[3].w)));
  }
  if (threadIdx.x == 0 && n_rows > 0)
    p.ends[at + c] = make_int4(any ? -1 : rows[0].x, rows[0].y, rows[n_rows - 1].x, rows[n_rows - 1].y);
  if (threadIdx.x == 0 && c == 0 && b == 0) p.head[0] = p.key;
  cluster_barrier();
  bool any_falls = false;
  for (int k = 0; k < blocks; ++k) {
    const int4 e = __ldcg(p.ends + at + k);
    any_falls |= e.x < 0;
    if (k + 1 < blocks) {
      const int4 next = __ldcg(p.ends + at + k + 1);
      any_falls |= next.x < e.z || next.y < e.w;  // (next.x -1 is seen when its turn comes)
    }
  }
  if (warp < kSmall / kTile) {
    const int n = c * (kSmall / kTile) + warp;
    int done = 0, m_lo = INT_MAX, m_hi = -1;
    if (n < p.n_t) {
      uint16_t *out = p.cols + (at + n) * p.n_t;
      for (int m0 = 0; m0 < p.n_t; m0 += 32) {
        const int m = m0 + lane;
        const int4 q = m < p.n_t ? __ldcg(p.tiles + at + m) : make_int4(INT_MAX, 0, INT_MAX, 0);
        const bool sees = tile_sees(q, n * kTile);
        const uint32_t bits = __ballot_sync(0xffffffffu, sees);
        if (sees) out[done + __popc(bits & ((1u << lane) - 1u))] = (uint16_t)(2 * m + tile_whole(q, n * kTile));
        if (bits) m_lo = min(m_lo, m0 + __ffs(bits) - 1), m_hi = m0 + 31 - __clz(bits);
        done += __popc(bits);
      }
      if (lane == 0) p.col_n[at + n] = done;
    }
    if (lane == 0) listed[warp] = make_int2(m_lo, m_hi);
  }
  __syncthreads();
  if (on) {
    const int2 m = listed[threadIdx.x / kTile];
    int2 q = make_int2(0, any_falls ? -1 : 0);
    if (!any_falls && m.y >= 0 && live) {
      const int2 *rg = p.ranges + (long long)b * p.Sp;
      const int lo = m.x * kTile, hi = min(m.y * kTile + kTile, p.S);
      q = queries_of(i, lo, hi, [&](int k) {
        const int2 r = __ldcg(rg + k);
        return make_int2(r.x, r.x + r.y);
      });
    }
    p.keys[(long long)b * p.Sp + i] = q;
  }
  cluster_barrier();
  if (mine < p.n_t) {
    const int n = __ldcg(p.col_n + at + mine);
    int rank = 0;
    for (int k = 0; k < p.n_t; ++k) {
      const int other = __ldcg(p.col_n + at + k);
      rank += other > n || (other == n && k < mine) ? 1 : 0;
    }
    p.order[at + rank] = make_int2(mine, n);
  }
}

// B (up to 65535), S (up to 2^22) and the causal flag as they are, under a mark
// that no zeroed buffer has.  (A hash of 32 bits took a plan of 257 rows of 1024
// tokens for one of 125184.)
uint64_t mask_key(const ulysses_problem &p) {
  return 0x6d61736bull << 40 | (uint64_t)p.B << 24 | (uint64_t)p.S << 1 | (uint64_t)p.causal;
}

}  // namespace

MaskLayout mask_layout(const ulysses_problem &p) {
  MaskLayout L;
  const size_t n_t = (size_t)(p.S + kTile - 1) / kTile, B = (size_t)p.B;
  L.ranges = 256;
  L.keys = L.ranges + up256(B * n_t * kTile * sizeof(int2));
  L.tiles = L.keys + up256(B * n_t * kTile * sizeof(int2));
  L.ends = L.tiles + up256(B * n_t * sizeof(int4));
  L.edges = L.ends + up256(B * n_t * sizeof(int4));
  L.col_n = L.edges + up256(B * n_t * sizeof(int2));
  L.cols = L.col_n + up256(B * n_t * sizeof(int));
  L.total = L.cols + up256(B * n_t * n_t * sizeof(uint16_t));
  return L;
}

dev::MaskView mask_view(const ulysses_problem &p, const void *mask) {
  dev::MaskView v{};
  if (!mask) return v;
  const MaskLayout L = mask_layout(p);
  const uint8_t *w = static_cast<const uint8_t *>(mask);
  v.n_t = (p.S + kTile - 1) / kTile;
  v.Sp = v.n_t * kTile;
  v.rows_n = (long long)p.B * v.Sp;
  v.ranges = reinterpret_cast<const int2 *>(w + L.ranges);
  v.keys = reinterpret_cast<const int2 *>(w + L.keys);
  v.tiles = reinterpret_cast<const int4 *>(w + L.tiles);
  v.col_n = reinterpret_cast<const int *>(w + L.col_n);
  v.cols = reinterpret_cast<const uint16_t *>(w + L.cols);
  v.order = reinterpret_cast<const int2 *>(w + L.edges);
  v.head = reinterpret_cast<const uint64_t *>(w);
  v.key = mask_key(p);
  return v;
}

cudaError_t launch_mask_build(const ulysses_problem &p, const int *doc, const int *prefix, int window, void *mask,
                              cudaStream_t st) {
  const MaskLayout L = mask_layout(p);
  uint8_t *w = static_cast<uint8_t *>(mask);
  BuildParams b{};
  b.doc = doc, b.prefix = prefix, b.window = window, b.causal = p.causal;
  b.S = p.S, b.n_t = (p.S + kTile - 1) / kTile, b.Sp = b.n_t * kTile;
  b.ranges = reinterpret_cast<int2 *>(w + L.ranges);
  b.keys = reinterpret_cast<int2 *>(w + L.keys);
  b.tiles = reinterpret_cast<int4 *>(w + L.tiles);
  b.ends = reinterpret_cast<int4 *>(w + L.ends);
  b.edges = reinterpret_cast<int2 *>(w + L.edges);
  b.order = reinterpret_cast<int2 *>(w + L.edges);  // (the edges have been read by then)
  b.col_n = reinterpret_cast<int *>(w + L.col_n);
  b.cols = reinterpret_cast<uint16_t *>(w + L.cols);
  b.head = reinterpret_cast<uint64_t *>(w);
  b.key = mask_key(p);
  if (p.S <= kSmall) {
    mask_small_kernel<<<(unsigned)p.B, kSmall, 0, st>>>(b);
    return cudaGetLastError();
  }
  cudaError_t e = cudaSuccess;
  if (p.S <= kMiddle) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.S <= 2 * kSmall ? 2 : p.S <= 4 * kSmall ? 4 : 8;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(attr[0].val.clusterDim.x, (unsigned)p.B);
    cfg.blockDim = dim3(kSmall);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mask_cluster_kernel, b);
  }
  const dim3 grid((unsigned)b.n_t, (unsigned)p.B);
  if (doc) {
    mask_edges_kernel<<<grid, kTile, 0, st>>>(b);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  mask_ranges_kernel<<<grid, kTile, 0, st>>>(b);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  mask_lists_kernel<<<grid, kTile, 0, st>>>(b);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  mask_order_kernel<<<(unsigned)p.B, 256, 0, st>>>(b);
  return cudaGetLastError();
}

}  // namespace ulysses
