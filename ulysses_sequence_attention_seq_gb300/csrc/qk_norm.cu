// qk_norm.cu -- RMS norm of every query and key head fused into the pack, and
// its backward.
//
// Models that normalise queries and keys do so per head, before the rotation
// ("Comparing Ulysses and Megatron Sequence Parallelism", "A simple attention
// skeleton": q, k viewed as heads, then rope, then the transpose).  For a head
// row x of D elements:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = rope(n * w)
// and y goes where the seq -> head All-to-All sends the row (permute.cu; v is
// copied).  Given g = dL/d(n * w), which is what the attention backward
// returns (it undoes the rotation):
//   dx = r * (g w - n * mean(g w n)),   dw = sum over rows of g n.
// Everything is float arithmetic on the stored values with one rounding to the
// element type per output.
//
// Both kernels move every byte once and do ~20 operations an element, so
// memory bandwidth is their bound.  A head row is held by D/16 (bf16) or D/8
// (fp32) consecutive lanes, each with the 16-byte chunk c of both halves: the
// rotation pair (i, i + D/2) is in one thread, a row's sums are shuffles over
// its lanes, and since a warp is a whole number of rows a thread keeps its c
// for the whole launch.
#include <atomic>

#include <cuda_bf16.h>
#include <stdint.h>

#include "check.cuh"
#include "internal.h"
#include "mask.cuh"
#include "sm100.cuh"

namespace ulysses {
namespace {

constexpr int kMaxDevices = 64;

using sm100::fma2;
using sm100::mul2;
using sm100::sub2;

// 16 bytes of T as pairs of floats, and back (one rounding).  The arithmetic
// below is on pairs: packed float instructions do two elements each.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int V = 8, N = 4;  // elements, pairs
  static __device__ __forceinline__ void load(const uint4 &u, float2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)  // a bf16 is the upper half of its float
      x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 store(const float2 (&x)[4]) {
    return make_uint4(sm100::pack_bf16x2(x[0].x, x[0].y), sm100::pack_bf16x2(x[1].x, x[1].y),
                      sm100::pack_bf16x2(x[2].x, x[2].y), sm100::pack_bf16x2(x[3].x, x[3].y));
  }
};
template <>
struct Vec<float> {
  static constexpr int V = 4, N = 2;
  static __device__ __forceinline__ void load(const uint4 &u, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 store(const float2 (&x)[2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  }
};

// n / d for 0 <= n < 2^31 by one multiplication (n * ceil(2^k / d) >> k with
// k = 31 + ceil(log2 d): exact for 31-bit n).
struct FastDiv {
  uint32_t mul, shift, d;
};
FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1u << s) < d) ++s;  // d <= 2^30
  const uint64_t k = 31 + s;
  return {(uint32_t)(((1ull << k) + d - 1) / d), (uint32_t)(k - 32), d};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
  return f.d == 1 ? n : __umulhi(n, f.mul) >> f.shift;
}

struct NormParams {
  const void *q, *k, *v;    // sequence layout
  const void *wq, *wk;      // [D] or null
  void *qo, *ko, *vo;       // forward: head layout
  const void *gq, *gk;      // backward: dL/d(n w), sequence layout
  void *dq, *dk;            // backward: sequence layout
  float *part;              // backward: [grid][2][D] partial weight gradients; with one block,
  float *dwq, *dwk;         // or without room for two, straight into these
  int P, B, Sl, D, H, KV, Pu, Cs, rep;
  float eps;
  int rope;
  FastDiv by_sl, by_b, by_pu;            // a token row's place
  FastDiv by_h, by_kv, by_qd, by_kd;     // heads of a row, heads a rank holds
  const float *cs, *sn;     // [S][D/2]
  uint32_t *status;
  uint32_t rope_key;
  dev::MaskView mask;       // rows that see nothing: written as zeros (null: none)
  long long q_n, k_n, qh_n, kh_n, rope_n, part_n;
};

// Token row (s*B + b)*Sl + t of the sequence layout.
struct RowPlace {
  int s, b, t;
};
__device__ __forceinline__ RowPlace place_of(const NormParams &p, long long row) {
  RowPlace r;
  if (row <= 0x7fffffffll) {
    const uint32_t sb = div_by((uint32_t)row, p.by_sl);
    r.t = (int)((uint32_t)row - sb * p.by_sl.d);
    r.s = (int)div_by(sb, p.by_b);
    r.b = (int)(sb - (uint32_t)r.s * p.by_b.d);
  } else {
    const long long sb = row / p.Sl;
    r.t = (int)(row - sb * p.Sl);
    r.s = (int)(sb / p.B);
    r.b = (int)(sb - (long long)r.s * p.B);
  }
  return r;
}

// What a warp takes at a time is a chunk, kPer (head, token) pairs for each of
// its groups of lanes.  Every warp has a ring of kStages chunks of its own,
// filled by bulk copies, so the copy engine and not registers holds the bytes
// in flight, and no warp waits for another.

// A warp's ring and its barriers, one a stage.
struct Ring {
  uint32_t smem, bar;
  volatile int *abort_flag;
  uint32_t *status;
};
__device__ __forceinline__ bool ring_wait(const Ring &r, int stage, int phase) {
  return __all_sync(0xffffffffu,
                    sm100::mbar_wait_bounded(r.bar + 8 * stage, (uint32_t)phase, r.abort_flag, r.status));
}
// After a failed wait: let the warp's copies in flight land before the block goes.
template <int kStages>
__device__ __forceinline__ void ring_drain(const Ring &r, long long done, long long issued) {
  volatile int never = 0;
  if ((threadIdx.x & 31) == 0) {
    atomicOr(r.status, (uint32_t)ULYSSES_STATUS_FWD_TIMEOUT);
    for (long long k = done; k < issued; ++k)
      sm100::mbar_wait_bounded(r.bar + 8 * (uint32_t)(k % kStages), (uint32_t)(k / kStages & 1), &never, nullptr,
                               200000000ull);
  }
  __syncwarp();
}

// The weights of q and k as floats, four at a time so that lanes c read
// neighbouring 16 bytes: [q, k][quad of a chunk][chunk c of the first half,
// then of the second].
template <typename T, int kThreads>
__device__ __forceinline__ void load_weights(const NormParams &p, float4 (&wts)[2][Vec<T>::N / 2][32]) {
  constexpr int V = Vec<T>::V;
  const int half = p.D / 2, lanes = half / V;
  for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
    const int which = i >= p.D, e = which ? i - p.D : i;
    const T *w = static_cast<const T *>(which ? p.wk : p.wq);
    const int h = e / half, cc = (e % half) / V, in = e % V;
    reinterpret_cast<float *>(&wts[which][in / 4][h * lanes + cc])[in % 4] = w ? (float)w[e] : 1.f;
  }
}
template <typename T>
__device__ __forceinline__ void weights_of(const float4 (&wts)[Vec<T>::N / 2][32], int at, float2 (&w)[Vec<T>::N]) {
#pragma unroll
  for (int e = 0; e < Vec<T>::N / 2; ++e) {
    const float4 v = wts[e][at];
    w[2 * e] = make_float2(v.x, v.y), w[2 * e + 1] = make_float2(v.z, v.w);
  }
}

// The forward.  A warp takes whole token rows (kMulti: several rows at once,
// where all their pairs fit one chunk): a row's heads of q, then k, then v are
// one list, cut into chunks.  What belongs to the row (its place on the head
// side, its cos and sin) is then found and loaded once for all its chunks.
// 32K tokens x 96 heads of 128: 265 us, 6.1 TB/s
// (blocks sharing one ring: 357 us, two barriers a chunk hold their warps
// together; rows cut into parts for more tasks: 275 us, and no faster at 8K
// tokens, 45 us).
template <typename T, int kWarps, int kStages, int kPer, bool kMulti>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_pack_kernel(const NormParams p, const int rows_per_task,
                                                                const int chunks_per_task) {
  constexpr int V = Vec<T>::V, N = Vec<T>::N;
  constexpr uint32_t kChunk = 1024 * kPer;
  extern __shared__ __align__(128) uint8_t stage_all[];  // [kWarps][kStages][kChunk]
  __shared__ __align__(16) float4 wts[2][N / 2][32];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ int aborted;
  if ((p.rope && p.status[1] != p.rope_key) || !dev::mask_matches(p.mask)) {
    if (blockIdx.x == 0 && threadIdx.x == 0)
      atomicOr(p.status, (uint32_t)(dev::mask_matches(p.mask) ? ULYSSES_STATUS_ROPE_TABLE : ULYSSES_STATUS_MASK));
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.D / 2, lanes = half / V;  // lanes <= 16
  const int c = lane % lanes, g0 = lane / lanes, groups = 32 / lanes, per = groups * kPer;
  const uint32_t pair_bytes = (uint32_t)(p.D * sizeof(T));
  const float inv_d = 1.0f / (float)p.D;
  const int H = p.H, KV = p.KV, np = H + 2 * KV;  // pairs of a row
  const long long rows = (long long)p.P * p.B * p.Sl;
  const long long tasks = (rows + rows_per_task - 1) / rows_per_task;
  uint8_t *stage = stage_all + warp * kStages * kChunk;
  const Ring ring = {sm100::smem_u32(stage), sm100::smem_u32(bars[warp]), &aborted, p.status};
  load_weights<T, 32 * kWarps>(p, wts);
  if (threadIdx.x == 0) aborted = 0;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) sm100::mbar_init(ring.bar + 8 * i, 1);
    sm100::fence_barrier_init();
  }
  __syncthreads();
  const long long w0 = (long long)blockIdx.x * kWarps + warp, stride = (long long)gridDim.x * kWarps;
  const long long mine = (tasks > w0 ? (tasks - 1 - w0) / stride + 1 : 0) * chunks_per_task;
  // Pairs [i0, i1) of `row`'s list into the ring at byte `at`; their bytes.
  auto load_pairs = [&](long long row, int i0, int i1, uint32_t at, uint32_t bar) {
    const int cut[4] = {0, H, H + KV, np};
#pragma unroll
    for (int w = 0; w < 3; ++w) {
      const int a = i0 > cut[w] ? i0 : cut[w], b = i1 < cut[w + 1] ? i1 : cut[w + 1];
      if (a >= b) continue;
      const long long off = (row * (w ? KV : H) + (a - cut[w])) * p.D;
      const T *src = static_cast<const T *>(w == 0 ? p.q : w == 1 ? p.k : p.v) + off;
      if (in_range(p.status, off, (long long)(b - a) * p.D, w ? p.k_n : p.q_n))
        sm100::bulk_load(at + (uint32_t)(a - i0) * pair_bytes, src, (uint32_t)(b - a) * pair_bytes, bar);
    }
  };
  long long next_task = w0;  // the next chunk to load
  int next_chunk = 0, next_stage = 0;
  auto load = [&]() {  // one lane issues, all keep count
    if (lane == 0) {
      const uint32_t bar = ring.bar + 8 * next_stage, at = ring.smem + next_stage * kChunk;
      const long long row = next_task * rows_per_task;
      if constexpr (kMulti) {
        const int nr = (int)(rows - row < rows_per_task ? rows - row : rows_per_task);
        sm100::mbar_arrive_expect_tx(bar, (uint32_t)(nr * np) * pair_bytes);
        for (int r = 0; r < nr; ++r) load_pairs(row + r, 0, np, at + (uint32_t)(r * np) * pair_bytes, bar);
      } else {
        const int i0 = next_chunk * per, i1 = i0 + per < np ? i0 + per : np;
        sm100::mbar_arrive_expect_tx(bar, (uint32_t)(i1 - i0) * pair_bytes);
        load_pairs(row, i0, i1, at, bar);
      }
    }
    if (++next_chunk == chunks_per_task) next_chunk = 0, next_task += stride;
    if (++next_stage == kStages) next_stage = 0;
  };
  long long issued = 0;
  for (; issued < kStages && issued < mine; ++issued) load();
  long long task = w0, first = 0;  // first: the row's place for rank d = 0 on the head side
  int chunk = 0, st = 0, phase = 0, dead = 0;
  bool live = true;
  float4 c4[N / 2], s4[N / 2];
  bool rot = false;
  for (long long k = 0; k < mine; ++k) {
    if (chunk == 0) {
      const long long row = task * rows_per_task + (kMulti ? g0 / np : 0);  // (kMulti: kPer is 1)
      live = row < rows && (!kMulti || g0 / np < rows_per_task);
      const RowPlace r = place_of(p, live ? row : 0);
      const int pos = r.s * p.Sl + r.t, rp = (int)div_by((uint32_t)r.s, p.by_pu);
      first = ((long long)rp * p.Pu * p.B + r.b) * p.Cs + (pos - rp * p.Cs);
      dead = dev::row_empty(p.mask, r.b, pos, p.status);
      const long long toff = (long long)pos * half + c * V;
      rot = p.rope && in_range(p.status, toff, V, p.rope_n);
      if (rot) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          c4[e] = __ldg(reinterpret_cast<const float4 *>(p.cs + toff + 4 * e));
          s4[e] = __ldg(reinterpret_cast<const float4 *>(p.sn + toff + 4 * e));
        }
      }
    }
    if (!ring_wait(ring, st, phase)) {
      ring_drain<kStages>(ring, k, issued);
      return;
    }
    uint4 a4[kPer], b4[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint8_t *sp = stage + st * kChunk + (uint32_t)(g0 + i * groups) * pair_bytes + c * 16;
      a4[i] = *reinterpret_cast<const uint4 *>(sp);
      b4[i] = *reinterpret_cast<const uint4 *>(sp + pair_bytes / 2);
    }
    __syncwarp();  // the stage has been read
    if (issued < mine) {
      load();
      ++issued;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int idx = kMulti ? g0 % np : chunk * per + g0 + i * groups;
      const int which = idx < H ? 0 : idx < H + KV ? 1 : 2;
      const int head = idx - (which == 0 ? 0 : which == 1 ? H : H + KV);
      if (dead) a4[i] = b4[i] = make_uint4(0u, 0u, 0u, 0u);
      float2 x[N], y[N], w[N];
      Vec<T>::load(a4[i], x);
      Vec<T>::load(b4[i], y);
      float2 s2 = make_float2(0.f, 0.f), t2 = s2;
#pragma unroll
      for (int e = 0; e < N; ++e) s2 = fma2(x[e], x[e], s2), t2 = fma2(y[e], y[e], t2);
      float ss = (s2.x + s2.y) + (t2.x + t2.y);
      for (int off = lanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (which < 2) {
        const float rn = rsqrtf(fmaf(ss, inv_d, p.eps));
        const float2 rr = make_float2(rn, rn);
        weights_of<T>(wts[which], c, w);
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = mul2(mul2(x[e], rr), w[e]);
        weights_of<T>(wts[which], lanes + c, w);
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] = mul2(mul2(y[e], rr), w[e]);
        if (rot) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float4 cq4 = c4[e / 2], sq4 = s4[e / 2];
            const float2 cc = e & 1 ? make_float2(cq4.z, cq4.w) : make_float2(cq4.x, cq4.y);
            const float2 sv = e & 1 ? make_float2(sq4.z, sq4.w) : make_float2(sq4.x, sq4.y);
            const float2 nx = sub2(mul2(x[e], cc), mul2(y[e], sv));
            y[e] = fma2(y[e], cc, mul2(x[e], sv));
            x[e] = nx;
          }
        }
        a4[i] = Vec<T>::store(x);
        b4[i] = Vec<T>::store(y);
      }
      if (!live || idx >= np) continue;
      // rank d of the token's ring position, local head j; a kv-head that
      // `rep` ranks read goes to each of them
      const int hd = which ? (int)p.by_kd.d : (int)p.by_qd.d, rep = which ? p.rep : 1;
      int d = (int)div_by((uint32_t)head, which ? p.by_kd : p.by_qd);
      const int j = head - d * hd;
      if (rep > 1) d = head * rep;  // (hd is 1)
      T *to = static_cast<T *>(which == 0 ? p.qo : which == 1 ? p.ko : p.vo);
      const long long rank = (long long)p.B * p.Cs;  // rows between two ranks
      long long o = (first + d * rank) * (long long)(hd * p.D) + j * p.D + c * V;
      for (int q = 0; q < rep; ++q, o += rank * p.D) {
        if (!in_range(p.status, o, half + V, which ? p.kh_n : p.qh_n)) continue;
        *reinterpret_cast<uint4 *>(to + o) = a4[i];
        *reinterpret_cast<uint4 *>(to + o + half) = b4[i];
      }
    }
    if (++chunk == chunks_per_task) chunk = 0, task += stride;
    if (++st == kStages) st = 0, phase ^= 1;
  }
}

// The backward: dx per row, and the block's share of both weight gradients.
// A warp takes its chunks of q, then those of k, a stage holding the same
// pairs of x and of g.  A thread adds its pairs' g n in a fixed order, the
// block its threads' in thread order and qk_norm_dw_kernel the blocks' in
// block order: dw does not vary from call to call (the grid depends on the
// device alone).  32K tokens x (32 + 32) heads of 128: 245 us, 6.6 TB/s (4
// warps a block 287 us, 1 KB chunks 300 us, 4 KB chunks 281 us).
template <typename T, int kWarps, int kStages, int kPer, bool kMask>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_bwd_kernel(const NormParams p) {
  constexpr int kThreads = 32 * kWarps;
  constexpr int V = Vec<T>::V, N = Vec<T>::N;
  constexpr uint32_t kChunk = 1024 * kPer;
  extern __shared__ __align__(128) uint8_t stage_all[];  // [kWarps][kStages][2][kChunk]
  __shared__ __align__(16) float4 wts[2][N / 2][32];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ int aborted;
  __shared__ float red[kThreads][2 * V + 1];
  if (!dev::mask_matches(p.mask)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, (uint32_t)ULYSSES_STATUS_MASK);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.D / 2, lanes = half / V;
  const int c = lane % lanes, g0 = lane / lanes, groups = 32 / lanes, per = groups * kPer;
  const float inv_d = 1.0f / (float)p.D;
  const long long rows = (long long)p.P * p.B * p.Sl;
  const long long nq = rows * p.H, nk = rows * p.KV;
  const long long cq = (nq + per - 1) / per, ck = (nk + per - 1) / per;
  uint8_t *stage = stage_all + warp * kStages * 2 * kChunk;
  const Ring ring = {sm100::smem_u32(stage), sm100::smem_u32(bars[warp]), &aborted, p.status};
  load_weights<T, 32 * kWarps>(p, wts);
  if (threadIdx.x == 0) aborted = 0;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) sm100::mbar_init(ring.bar + 8 * i, 1);
    sm100::fence_barrier_init();
  }
  __syncthreads();
  // this warp's chunks: mq of q, then the rest of k
  const long long w0 = (long long)blockIdx.x * kWarps + warp, stride = (long long)gridDim.x * kWarps;
  const long long mq = cq > w0 ? (cq - 1 - w0) / stride + 1 : 0;
  const long long mine = mq + (ck > w0 ? (ck - 1 - w0) / stride + 1 : 0);
  auto load = [&](long long k) {  // one lane
    const bool which = k >= mq;
    const long long first = (w0 + (which ? k - mq : k) * stride) * per;
    const long long left = (which ? nk : nq) - first;
    const uint32_t bytes = (uint32_t)(left < per ? left : per) * (uint32_t)(p.D * sizeof(T));
    const int st = (int)(k % kStages);
    sm100::mbar_arrive_expect_tx(ring.bar + 8 * st, 2 * bytes);
    if (!in_range(p.status, first * p.D, bytes / sizeof(T), which ? p.k_n : p.q_n)) return;
    const uint32_t dst = ring.smem + st * 2 * kChunk;
    sm100::bulk_load(dst, static_cast<const T *>(which ? p.k : p.q) + first * p.D, bytes, ring.bar + 8 * st);
    sm100::bulk_load(dst + kChunk, static_cast<const T *>(which ? p.gk : p.gq) + first * p.D, bytes,
                     ring.bar + 8 * st);
  };
  long long issued = 0;
  for (; issued < kStages && issued < mine; ++issued)
    if (lane == 0) load(issued);
  bool fine = true;
  auto step = [&](long long k, int which, float2 (&a0)[N], float2 (&a1)[N]) -> bool {
    const int st = (int)(k % kStages);
    const long long first = (w0 + (which ? k - mq : k) * stride) * per, n = which ? nk : nq;
    if (!ring_wait(ring, st, (int)(k / kStages & 1))) {
      ring_drain<kStages>(ring, k, issued);
      return false;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint8_t *sp = stage + st * 2 * kChunk + (uint32_t)((g0 + i * groups) * p.D + c * V) * (uint32_t)sizeof(T);
      uint4 xa = *reinterpret_cast<const uint4 *>(sp), xb = *reinterpret_cast<const uint4 *>(sp + half * sizeof(T));
      uint4 ga = *reinterpret_cast<const uint4 *>(sp + kChunk);
      uint4 gb = *reinterpret_cast<const uint4 *>(sp + kChunk + half * sizeof(T));
      const long long it = first + g0 + i * groups;
      bool dead = it >= n;
      if (kMask && !dead) {
        const FastDiv &by = which ? p.by_kv : p.by_h;
        const RowPlace r = place_of(p, it <= 0x7fffffffll ? (long long)div_by((uint32_t)it, by) : it / by.d);
        dead = dev::row_empty(p.mask, r.b, r.s * p.Sl + r.t, p.status);
      }
      if (dead) xa = xb = ga = gb = make_uint4(0u, 0u, 0u, 0u);
      float2 x0[N], x1[N], y0[N], y1[N], wx[N], wy[N];
      Vec<T>::load(xa, x0);
      Vec<T>::load(xb, x1);
      Vec<T>::load(ga, y0);
      Vec<T>::load(gb, y1);
      weights_of<T>(wts[which], c, wx);
      weights_of<T>(wts[which], lanes + c, wy);
      float2 s2 = make_float2(0.f, 0.f), t2 = s2;  // sum x^2, sum g w x
#pragma unroll
      for (int e = 0; e < N; ++e) {
        wx[e] = mul2(y0[e], wx[e]), wy[e] = mul2(y1[e], wy[e]);  // g w
        s2 = fma2(x0[e], x0[e], fma2(x1[e], x1[e], s2));
        t2 = fma2(wx[e], x0[e], fma2(wy[e], x1[e], t2));
      }
      float ss = s2.x + s2.y, gx = t2.x + t2.y;
      for (int off = lanes / 2; off > 0; off >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, off);
        gx += __shfl_xor_sync(0xffffffffu, gx, off);
      }
      const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
      const float m = -gx * r * r * inv_d;  // n * mean(g w n) = x r * (r gx / D) = r (-x m)
      const float2 rr = make_float2(r, r), mm = make_float2(m, m);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        a0[e] = fma2(y0[e], mul2(x0[e], rr), a0[e]);
        a1[e] = fma2(y1[e], mul2(x1[e], rr), a1[e]);
        x0[e] = mul2(rr, fma2(x0[e], mm, wx[e]));
        x1[e] = mul2(rr, fma2(x1[e], mm, wy[e]));
      }
      const long long o = it * p.D + c * V;
      if (it < n && in_range(p.status, o, half + V, which ? p.k_n : p.q_n)) {
        T *dst = static_cast<T *>(which ? p.dk : p.dq) + o;
        *reinterpret_cast<uint4 *>(dst) = Vec<T>::store(x0);
        *reinterpret_cast<uint4 *>(dst + half) = Vec<T>::store(x1);
      }
    }
    __syncwarp();  // the stage has been read
    if (issued < mine) {
      if (lane == 0) load(issued);
      ++issued;
    }
    return true;
  };
  long long k = 0;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float2 a0[N], a1[N];  // the weight's gradient so far
#pragma unroll
    for (int e = 0; e < N; ++e) a0[e] = a1[e] = make_float2(0.f, 0.f);
    for (; fine && k < (which ? mine : mq); ++k) fine = step(k, which, a0, a1);
    if (__syncthreads_or(!fine)) return;  // (the first half's sums have been read, too)
    if (!(which ? p.dwk : p.dwq)) continue;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      red[threadIdx.x][2 * e] = a0[e].x, red[threadIdx.x][2 * e + 1] = a0[e].y;
      red[threadIdx.x][V + 2 * e] = a1[e].x, red[threadIdx.x][V + 2 * e + 1] = a1[e].y;
    }
    __syncthreads();
    // element e of the row: chunk cc = (e % half) / V of half e / half
    for (int e = threadIdx.x; e < p.D; e += kThreads) {
      const int cc = (e % half) / V, i = (e / half) * V + e % V;
      float sum = 0.f;
      for (int th = cc; th < kThreads; th += lanes) sum += red[th][i];
      if (gridDim.x > 1) {
        const long long at = ((long long)blockIdx.x * 2 + which) * p.D + e;
        if (in_range(p.status, at, 1, p.part_n)) p.part[at] = sum;
      } else {
        (which ? p.dwk : p.dwq)[e] = sum;
      }
    }
  }
}

// dw[which][e] = sum over the blocks' partials: 32 columns a block, 32 threads
// a column.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float *__restrict__ part, int n_part, int D, float *dwq,
                                                          float *dwk) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;  // which * D + e
  float sum = 0.f;
  for (int i = threadIdx.y; i < n_part; i += 32) sum += part[(long long)i * 2 * D + col];
  red[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0) {
    sum = 0.f;
    for (int i = 0; i < 32; ++i) sum += red[i][threadIdx.x];
    float *dst = col < D ? dwq : dwk;
    if (dst) dst[col < D ? col : col - D] = sum;
  }
}

NormParams params_of(const ulysses_problem &p, const void *ws, float eps, const void *mask) {
  NormParams n{};
  const WorkspaceLayout L = workspace_layout(p);
  const uint8_t *w = static_cast<const uint8_t *>(ws);
  n.P = p.P, n.B = p.B, n.Sl = p.S / p.P, n.D = p.head_dim, n.H = p.n_head, n.KV = p.n_kv_head;
  n.Pu = group_ranks(p), n.Cs = chunk_len(p), n.rep = kv_replicas(p);
  n.eps = eps;
  n.rope = p.use_rope;
  n.cs = reinterpret_cast<const float *>(w + L.rope);
  n.sn = n.cs + (size_t)p.S * (p.head_dim / 2);
  n.status = reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(w + L.status));
  n.rope_key = rope_key(p);
  n.mask = mask_view(p, mask);
  n.q_n = (long long)p.B * p.S * p.n_head * p.head_dim;
  n.k_n = (long long)p.B * p.S * p.n_kv_head * p.head_dim;
  n.qh_n = n.q_n;
  n.kh_n = (long long)p.P * p.B * n.Cs * kv_per_rank(p) * p.head_dim;
  n.rope_n = (long long)p.S * (p.head_dim / 2);
  n.by_sl = fast_div((uint32_t)n.Sl);
  n.by_b = fast_div((uint32_t)n.B);
  n.by_pu = fast_div((uint32_t)n.Pu);
  n.by_h = fast_div((uint32_t)n.H);
  n.by_kv = fast_div((uint32_t)n.KV);
  return n;
}

// The blocks that are resident at once (asked once per kernel and device, when
// the kernel is also told its dynamic shared memory), and no more than `work`.
template <typename K>
cudaError_t resident_grid(K kernel, std::atomic<int> (&cache)[kMaxDevices], int threads, size_t smem, long long work,
                          int *grid) {
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices) n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int sms = 0, per = 0;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem)) != cudaSuccess)
      return e;
    n = sms * (per < 1 ? 1 : per);
    if (dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
  }
  *grid = (int)(work < n ? (work < 1 ? 1 : work) : n);
  return cudaSuccess;
}

template <typename T, int kPer, bool kMulti>
cudaError_t launch_fwd_as(const NormParams &n, long long rows, int rows_per_task, cudaStream_t st) {
  static std::atomic<int> cache[kMaxDevices];
  constexpr int kWarps = 4, kStages = 4;
  constexpr size_t smem = (size_t)kWarps * kStages * 1024 * kPer;
  const int per = kPer * 32 / (n.D / (2 * Vec<T>::V));
  const int chunks = kMulti ? 1 : (n.H + 2 * n.KV + per - 1) / per;
  const long long tasks = (rows + rows_per_task - 1) / rows_per_task;
  int grid = 0;
  const auto kernel = qk_norm_pack_kernel<T, kWarps, kStages, kPer, kMulti>;
  const cudaError_t e = resident_grid(kernel, cache, 32 * kWarps, smem, (tasks + kWarps - 1) / kWarps, &grid);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 32 * kWarps, smem, st>>>(n, rows_per_task, chunks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_fwd(const ulysses_problem &p, NormParams n, cudaStream_t st) {
  n.by_qd = fast_div((uint32_t)(p.n_head / n.Pu));
  n.by_kd = fast_div((uint32_t)kv_per_rank(p));
  const long long rows = (long long)p.B * p.S;
  const int groups = 32 / (p.head_dim / (2 * Vec<T>::V)), np = p.n_head + 2 * p.n_kv_head;
  // Two pairs a lane where a row fills that; one where it does not; several
  // rows a chunk where a row does not fill half of one.
  if (np >= 2 * groups) return launch_fwd_as<T, 2, false>(n, rows, 1, st);
  if (2 * np > groups) return launch_fwd_as<T, 1, false>(n, rows, 1, st);
  return launch_fwd_as<T, 1, true>(n, rows, groups / np, st);
}

template <typename T, bool kMask>
cudaError_t launch_bwd_as(const ulysses_problem &p, NormParams n, float *dwq, float *dwk, long long max_parts,
                          cudaStream_t st) {
  static std::atomic<int> cache[kMaxDevices];
  constexpr int kWarps = 8, kStages = 3, kPer = 2;
  constexpr size_t smem = (size_t)kWarps * kStages * 2 * 1024 * kPer;
  const int per = kPer * 32 / (p.head_dim / (2 * Vec<T>::V));
  const long long most = (long long)p.B * p.S * (p.n_head > p.n_kv_head ? p.n_head : p.n_kv_head);
  long long work = (most + (long long)per * kWarps - 1) / ((long long)per * kWarps);
  const bool dw = dwq || dwk;
  if (dw && work > max_parts) work = max_parts > 1 ? max_parts : 1;
  n.dwq = dwq, n.dwk = dwk;
  int grid = 0;
  const auto kernel = qk_norm_bwd_kernel<T, kWarps, kStages, kPer, kMask>;
  cudaError_t e = resident_grid(kernel, cache, 32 * kWarps, smem, work, &grid);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 32 * kWarps, smem, st>>>(n);
  e = cudaGetLastError();
  if (e != cudaSuccess || !dw || grid == 1) return e;
  qk_norm_dw_kernel<<<2 * p.head_dim / 32, dim3(32, 32), 0, st>>>(n.part, grid, p.head_dim, dwq, dwk);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const ulysses_problem &p, const NormParams &n, float *dwq, float *dwk, long long max_parts,
                       cudaStream_t st) {
  return n.mask.ranges ? launch_bwd_as<T, true>(p, n, dwq, dwk, max_parts, st)
                       : launch_bwd_as<T, false>(p, n, dwq, dwk, max_parts, st);
}

}  // namespace

cudaError_t launch_qk_norm_pack(const ulysses_problem &p, const void *q, const void *k, const void *v, const void *wq,
                                const void *wk, float eps, const void *mask, void *qh, void *kh, void *vh, void *ws,
                                cudaStream_t st) {
  NormParams n = params_of(p, ws, eps, mask);
  n.q = q, n.k = k, n.v = v, n.wq = wq, n.wk = wk, n.qo = qh, n.ko = kh, n.vo = vh;
  return p.dtype == ULYSSES_BF16 ? launch_fwd<__nv_bfloat16>(p, n, st) : launch_fwd<float>(p, n, st);
}

cudaError_t launch_qk_norm_bwd(const ulysses_problem &p, const void *q, const void *k, const void *wq, const void *wk,
                               float eps, const void *mask, const void *gq, const void *gk, void *dq, void *dk,
                               float *dwq, float *dwk, void *ws, cudaStream_t st) {
  NormParams n = params_of(p, ws, eps, mask);
  n.q = q, n.k = k, n.wq = wq, n.wk = wk, n.gq = gq, n.gk = gk, n.dq = dq, n.dk = dk;
  // The partial sums (2 D floats a block) live where the attention backward
  // keeps its copy of dO: that call is over by now.
  const WorkspaceLayout L = workspace_layout(p);
  const long long max_parts = (long long)((L.total_bwd - L.dohead) / ((size_t)2 * p.head_dim * 4));
  n.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + L.dohead);
  n.part_n = (long long)((L.total_bwd - L.dohead) / sizeof(float));
  return p.dtype == ULYSSES_BF16 ? launch_bwd<__nv_bfloat16>(p, n, dwq, dwk, max_parts, st)
                                 : launch_bwd<float>(p, n, dwq, dwk, max_parts, st);
}

}  // namespace ulysses
