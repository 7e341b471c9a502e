// attn_bwd_mod_tc.cu -- bf16 attention backward with modified scores on the
// 5th-generation tensor cores, the reverse All-to-All of the gradients fused
// into the epilogues.
//
// With the scores of score_mod.cuh, P = exp(x - lse) and f = 1 - tanh^2(s / cap)
// (1 without a cap):
//   dV = P^T dO          dP = dO V^T          dS = P f (dP - delta)
//   dQ = scale dS K      dK = scale dS^T Q    (dK, dV summed over the q-heads
//                                              that share a kv-head)
// The plain backward's two kernels (attn_bwd_tc.cu): dK/dV with one CTA per
// 128-key tile of a kv-head, dQ with one per 128-query tile of a q-head, same
// tiles, TMEM layout, rings and order of products, no atomics.  What differs:
//   - dK/dV runs over the query tiles that see its key tile (the mask plan's
//     list), dQ over the hull of what its rows see; tiles that see or are seen
//     by nothing write zeros.
//   - A tile that needs masking has P set to 0 outside an interval that each
//     thread holds in two registers: of keys where it owns a query (dQ), of
//     queries where it owns a key (dK/dV; the plan's key intervals, or where it
//     has none, each query's interval read from it).  Queries that see nothing
//     need no masking: their nlse is -inf.
//   - P and P f come from the raw scores in the forms of score_mod.cuh; a warp
//     runs its loop in one form until a tile needs a further one, and goes on
//     with that tile in the loop of that form, and a step is a step of masked or
//     of unmasked scores to its end.  Forms and masks inside one step cost 4
//     register moves a pair of scores where they met again.
//   - The softmax warps get 224 registers (with the plain dK/dV's 168 the cap's
//     coefficients spilled), the others 56: the issuer forms its descriptors at
//     each burst (32K tokens x 8 heads, capped: 6000 -> 5700 us for the two).
//   - dK/dV takes its key tiles in the plan's order, those with most query tiles
//     first: the items are few and differ, and the last to start set the end
//     (8K tokens x 32 heads in documents of about 2048: 688 -> 633 us).
//   - dQ's blocks go on with items of blocks that have not started
//     (work_items.cuh): the next rows of Q and dO go to tensor memory, and its
//     first S and dP are formed, during this item's epilogue.  8K tokens x 32
//     heads of 128 in equal documents of 1024: dQ 185 -> 161 us.  (dK/dV has 3.4 items
//     an SM there, four times as long each, and its K and V tiles fill shared
//     memory to the end of an item.)
// What bounds them is, as in the plain kernels, the chain from scores to P to dS
// and back to the tensor core, with some 190 instructions a step more in each
// warp for a capped score.  32K tokens x 8 heads of 128, causal, capped at 50:
// 5700 us, of which the packing of dO 85 (0.71 of the measured bf16 rate for the
// 7 products); 8K tokens x 32 heads in documents of about 2048, capped at 50:
// 602 us, mask only 519 us (617 us where they lie less well).
#include <cuda_bf16.h>
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

constexpr int kTmaWarp = 8, kMmaWarp = 9;
// Both kernels: warpgroups 0-1 softmax, warpgroup 2: TMA, MMA, 2 idle warps.
constexpr int kThreads = 384;
constexpr uint32_t kRegsProducer = 56, kRegsSoftmax = 224;
static_assert(128 * kRegsProducer + 256 * kRegsSoftmax <= 384 * 168, "register split over budget");
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
  int B, S, Sl, hp, kvp, group, causal;
  int n_head, n_kv;                    // global head counts (row widths of the seq layout)
  int group_kv, group_q;               // heads per CTA group (grouped_order) of the two kernels
  float scale, scale_log2;
  const float *nlse, *delta;           // [P][B][hp] rows of Cs values, Ld apart; nlse = -lse * log2(e)
  const float *rope_cos, *rope_sin;    // [S][D/2], or null without RoPE
  const __nv_bfloat16 *q, *dout;       // head layout [P][B][Cs][hp][D] (the dQ kernel's TMEM operands)
  __nv_bfloat16 *dq, *dk, *dv;         // sequence-sharded outputs
  int dq_by32, qo_by32;                // dq, and q and dout, lie on 32-byte boundaries
  int kv_rep;                          // > 1: replicated kv-heads; dk/dv then point to float
                                       // per-rank partials [P*B][Cs][D] (unscaled, not rotated)
  uint32_t *status;                    // status word; the RoPE table key follows it
  uint32_t rope_key;
  int Pu, Cs;                          // ranks of a ring position, tokens of its chunk (plain Ulysses: P, S)
  int Ld;                              // row stride of nlse / delta
  // Elements of the buffers read or written with plain loads and stores (range
  // checks of a checked build): dQ, dK / dV (or their float partials), Q / dO in
  // head layout, the nlse / delta rows, the RoPE table.
  long long dq_n, dkv_n, qo_n, rows_n, rope_n;
  dev::ScoreMod mod;
};

// Head-layout (rank * B + batch) of the rows at global position `pos` for the
// CTA of member*B + batch = `rb`.
__device__ __forceinline__ int hl_outer(const BwdParams &p, int rb, int pos) {
  return (pos / p.Cs) * p.Pu * p.B + rb;
}

// What a block looks at before it starts: the status word, the RoPE table's key
// and the plan's key, read together (each is a trip to L2).
struct Checks {
  uint32_t status, rope;
  uint64_t mask;
  __device__ __forceinline__ explicit Checks(const BwdParams &p) {
    const volatile uint32_t *st = p.status;
    status = st[0], rope = st[1], mask = dev::mask_key_of(p.mod.mask);
  }
  // False (and the status bit set) where an earlier kernel timed out or the table
  // or the plan belongs to another problem: the block then writes nothing.
  __device__ __forceinline__ bool fine(const BwdParams &p) const {
    const bool stale = p.rope_cos && rope != p.rope_key, other = mask != p.mod.mask.key && p.mod.mask.ranges;
    if (status & 3u) return false;
    if ((stale || other) && threadIdx.x == 0)
      atomicOr(p.status, (uint32_t)(stale ? ULYSSES_STATUS_ROPE_TABLE : ULYSSES_STATUS_MASK));
    return !stale && !other;
  }
};

// A descriptor formed where it stands: those of a burst are one addition each from
// it, and none is kept (and spilled) from one burst to the next.
__device__ __forceinline__ uint64_t here(uint64_t desc) {
  asm volatile("" : "+l"(desc));
  return desc;
}

// 32 fp32 accumulator columns -> scaled bf16 in global memory.
__device__ __forceinline__ void store_plain(__nv_bfloat16 *dst, const uint32_t (&x)[32], float scale) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e)
    w[e] = pack_bf16x2(__uint_as_float(x[2 * e]) * scale, __uint_as_float(x[2 * e + 1]) * scale);
  uint4 *d = reinterpret_cast<uint4 *>(dst);
#pragma unroll
  for (int v = 0; v < 4; ++v) d[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
}

// The cos / sin of rotation pairs [i0, i0+32) at one position, read ahead of
// the epilogue that undoes the rotation: `rope_prefetch` asks L2 for the two
// 128-byte rows (kept with evict-last priority: every head's CTAs over the
// same rows read them) when a CTA starts, `rope_load` brings them into
// registers while the last products are still running.
struct RopeRow {
  float4 c[8], s[8];
};
__device__ __forceinline__ void rope_prefetch(const float *cs, const float *sn) {
  asm volatile("prefetch.global.L2::evict_last [%0];" ::"l"(cs));
  asm volatile("prefetch.global.L2::evict_last [%0];" ::"l"(sn));
}
__device__ __forceinline__ void rope_load(RopeRow &a, const float *cs, const float *sn) {
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    a.c[v] = __ldg(reinterpret_cast<const float4 *>(cs) + v);
    a.s[v] = __ldg(reinterpret_cast<const float4 *>(sn) + v);
  }
}

// The same 16 pairs at a time, for the dQ kernel, whose items share their
// registers with an epilogue.
struct RopeHalf {
  float4 c[4], s[4];
};
__device__ __forceinline__ void rope_load(RopeHalf &a, const float *cs, const float *sn) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    a.c[v] = __ldg(reinterpret_cast<const float4 *>(cs) + v);
    a.s[v] = __ldg(reinterpret_cast<const float4 *>(sn) + v);
  }
}
__device__ __forceinline__ void store_unrotated(__nv_bfloat16 *dx, __nv_bfloat16 *dy, const uint32_t (&x)[16],
                                                const uint32_t (&y)[16], float scale, bool rot, const RopeHalf &a,
                                                bool by32) {
  uint32_t wx[8], wy[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float4 c4 = a.c[e / 2], s4 = a.s[e / 2];
    const float2 cc = e % 2 ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
    const float2 ss = e % 2 ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
    float2 u = make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
    float2 v = make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
    if (rot) {
      const float2 u0 = u;
      u = make_float2(u0.x * cc.x + v.x * ss.x, u0.y * cc.y + v.y * ss.y);
      v = make_float2(v.x * cc.x - u0.x * ss.x, v.y * cc.y - u0.y * ss.y);
    }
    wx[e] = pack_bf16x2(u.x * scale, u.y * scale);
    wy[e] = pack_bf16x2(v.x * scale, v.y * scale);
  }
  if (by32) {
    st_global_32(dx, wx);
    st_global_32(dy, wy);
  } else {
    uint4 *px = reinterpret_cast<uint4 *>(dx), *py = reinterpret_cast<uint4 *>(dy);
    px[0] = make_uint4(wx[0], wx[1], wx[2], wx[3]), px[1] = make_uint4(wx[4], wx[5], wx[6], wx[7]);
    py[0] = make_uint4(wy[0], wy[1], wy[2], wy[3]), py[1] = make_uint4(wy[4], wy[5], wy[6], wy[7]);
  }
}

// Columns [i0, i0+32) (x) and [i0+D/2, i0+D/2+32) (y) of a gradient row:
// scale, undo the rotation by the position's angle (x' = x cos + y sin,
// y' = y cos - x sin) when `rot`, round to bf16 and store.
__device__ __forceinline__ void store_unrotated(__nv_bfloat16 *dx, __nv_bfloat16 *dy, uint32_t (&x)[32],
                                                uint32_t (&y)[32], float scale, bool rot, const RopeRow &a) {
  if (rot) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 c4 = a.c[e / 4];
      const float4 s4 = a.s[e / 4];
      const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float a = __uint_as_float(x[e + q]), b = __uint_as_float(y[e + q]);
        x[e + q] = __float_as_uint(a * cc[q] + b * ss[q]);
        y[e + q] = __float_as_uint(b * cc[q] - a * ss[q]);
      }
    }
  }
  store_plain(dx, x, scale);
  store_plain(dy, y, scale);
}

// P (packed to bf16 in w where kPack) and what dS takes of it, pf = P f, from a
// thread's 64 raw scores: tanh in form kForm; the exponent offset -lse log2(e)
// of pair c from nl(c); `lead` as in dev::logits, the bias taken as linear
// where kLinear; with kMask, columns outside [lo, lo + len) are 0.  Returns the
// largest square of a score where the form depends on it.
template <int kMod, int kForm, bool kLinear, bool kPack, bool kMask, typename Form, typename Offset>
__device__ __forceinline__ float p_mod_as(const uint32_t (&s)[2][32], const Form &form, float sl,
                                          const dev::LinearBias &lb, float slope2, int lead, Offset nl, int lo, int len,
                                          float2 (&pf)[32], uint32_t (&w)[2][16]) {
  using namespace dev;
  constexpr bool kCap = (kMod & kModCap) != 0, kBias = (kMod & kModBias) != 0;
  const BiasSteps steps(lb);
  const f2x scale2 = f2_of(sl, sl);
  float bg[2] = {0.f, 0.f};
  const uint32_t seen[2] = {bits_of(lo, lo + len), bits_of(lo - 32, lo - 32 + len)};
#pragma unroll
  for (int c2 = 0; c2 < 32; c2 += 2) {
    const uint32_t *r = &s[c2 >> 4][2 * (c2 & 15)];
    f2x v[2] = {f2_of(__uint_as_float(r[0]), __uint_as_float(r[1])),
                f2_of(__uint_as_float(r[2]), __uint_as_float(r[3]))};
    if constexpr (kCap && kForm == 2) form.any(v[0], v[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c2 + h;
      f2x add = nl(c);
      if constexpr (kBias && kLinear) {
        const float b16 = fmaf((float)((c >> 3) * 16), lb.slope2, lb.base);
        add = f2_add(add, f2_add(steps.d[c & 7], f2_of(b16, b16)));
      }
      if constexpr (kBias && !kLinear)
        add = f2_add(add, f2_of(-slope2 * fabsf((float)(lead + 2 * c)), -slope2 * fabsf((float)(lead + 2 * c + 1))));
      f2x x, f;
      if constexpr (!kCap) {
        x = f2_fma(v[h], scale2, add);
      } else if constexpr (kForm < 2) {
        const f2x u = f2_mul(v[h], v[h]);
        if constexpr (kPack) {
          const float2 u2 = f2_to(u);
          bg[h] = max3(bg[h], u2.x, u2.y);
        }
        if constexpr (kForm == 0) {
          x = f2_fma(v[h], form.poly(u), add);
          f = form.slope(u);
        } else {
          v[h] = f2_mul(v[h], form.poly(u));
        }
      }
      if constexpr (kCap && kForm > 0) {
        x = f2_add(v[h], add);
        f = f2_fma(f2_mul(v[h], form.inv), f2_mul(v[h], form.ninv), form.one);
      }
      const float2 x2 = f2_to(x);
      float2 pe = make_float2(ex2(x2.x), ex2(x2.y));
      if constexpr (kMask) {
        if (!(seen[c >> 4] & (1u << (2 * (c & 15))))) pe.x = 0.f;
        if (!(seen[c >> 4] & (2u << (2 * (c & 15))))) pe.y = 0.f;
      }
      if constexpr (kPack) w[c >> 4][c & 15] = pack_bf16x2(pe.x, pe.y);
      if constexpr (kCap)
        pf[c] = f2_to(f2_mul(f2_of(pe.x, pe.y), f));
      else
        pf[c] = pe;
    }
  }
  return fmaxf(bg[0], bg[1]);
}
// The same with the bias's two cases: linear where all pairs of the warp lie on
// one side of the diagonal, or (`side`) all that are seen do.
template <int kMod, int kForm, bool kPack, bool kMask, typename Form, typename Offset>
__device__ __forceinline__ float p_mod(const uint32_t (&s)[2][32], const Form &form, float sl, float slope2,
                                       int lead, int side, Offset nl, int lo, int len, float2 (&pf)[32],
                                       uint32_t (&w)[2][16]) {
  dev::LinearBias lb{true, 0.f, 0.f};
  if constexpr ((kMod & kModBias) != 0) {
    lb = dev::linear_bias<64>(slope2, lead, side);
    if (!lb.ok) return p_mod_as<kMod, kForm, false, kPack, kMask>(s, form, sl, lb, slope2, lead, nl, lo, len, pf, w);
  }
  return p_mod_as<kMod, kForm, true, kPack, kMask>(s, form, sl, lb, slope2, lead, nl, lo, len, pf, w);
}

// dS = P * (dP - delta) for the same 64 columns (query c's delta at dl[c/2]).
__device__ __forceinline__ void ds_columns(const uint32_t (&d)[2][32], const float2 *dl, const float2 (&pf)[32],
                                           uint32_t (&w)[2][16]) {
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const uint32_t *dh = d[c >> 4];
    const float2 x = sub2(make_float2(__uint_as_float(dh[2 * (c & 15)]), __uint_as_float(dh[2 * (c & 15) + 1])),
                          dl[c]);
    const float2 ds = mul2(pf[c], x);
    w[c >> 4][c & 15] = pack_bf16x2(ds.x, ds.y);
  }
}

// ============================================================= dK / dV kernel
// (TMEM and rings as in attn_bwd_tc.cu.)
constexpr int kQSlots = 3, kOSlots = 2;

enum : uint32_t {
  kKBarIn = 0,
  kKBarQFull = 8,    // [3]
  kKBarQEmpty = 32,  // [3]
  kKBarOFull = 56,   // [2]
  kKBarOEmpty = 72,  // [2]
  kKBarSFull = 88,
  kKBarDPFull = 96,
  kKBarPFull = 104,  // 256 arrivals
  kKBarDSFull = 112, // 256 arrivals
  kKBarAcc = 120,
  kKBarDrain = 128,
  kKTmemSlot = 136,
  kKAbortSlot = 140,
  kKBarBytes = 144
};

constexpr uint32_t kMaxDynSmem = 232448;  // 227 KB per block

template <int D>
struct KVLayout {
  static constexpr uint32_t kT = 128u * D * 2;  // one 128-row tile
  static constexpr uint32_t oK = 0, oV = kT, oQ = 2 * kT, odO = oQ + kQSlots * kT,
                            oDl = odO + kOSlots * kT,  // delta rows, one per Q slot
                            oL = oDl + kQSlots * 512,  // -LSE*log2(e) rows, one per dO slot
                            oBar = oL + kOSlots * 512;
  static constexpr uint32_t kUsed = oBar + kKBarBytes;
  // Room for aligning the base to 1024 bytes where it fits; at D = 128 it
  // does not, and the kernel checks the base it was given.
  static constexpr uint32_t kAlloc = kUsed + 1024 <= kMaxDynSmem ? kUsed + 1024 : kMaxDynSmem;
  static_assert(kUsed <= kMaxDynSmem, "dK/dV tiles exceed shared memory");
};

template <int D, int kMod>
__global__ void __launch_bounds__(kThreads, 1)
    dkdv_mod_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                    const __grid_constant__ CUtensorMap tmL, const __grid_constant__ CUtensorMap tmDl,
                    const BwdParams p) {
  using L = KVLayout<D>;
  constexpr int kCh = D / 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t *smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const uint32_t sK = sb + L::oK, sV = sb + L::oV, sQ = sb + L::oQ, sdO = sb + L::odO,
                 sL = sb + L::oL, sDl = sb + L::oDl, bar = sb + L::oBar;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::oBar + kKAbortSlot);
  const volatile uint32_t *gst = p.status;
  const Checks checks(p);
  const int n_qt = (p.S + 127) / 128;
  const dev::HeadTile ht = dev::grouped_order((int)blockIdx.x, p.Pu * p.B * p.kvp, n_qt, p.group_kv);
  const int hid = ht.head;
  const int kl = hid % p.kvp, rb = hid / p.kvp;
  // the key tile (low ones have the most work under the causal flag), its query tiles
  int2 mine = make_int2(ht.rank, p.causal ? n_qt - ht.rank : n_qt);
  if (p.mod.mask.ranges) mine = dev::order_at(p.mod.mask, (long long)(rb % p.B) * n_qt + ht.rank, p.status);
  if (!checks.fine(p)) return;
  if (pad + L::kUsed > L::kAlloc) {  // uniform over the block: nobody has touched a barrier yet
    if (threadIdx.x == 0) atomicOr(p.status, (uint32_t)ULYSSES_STATUS_SMEM_ALIGN);
    return;
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = mine.x, n_m = mine.y;
  // mask plan: 2 * query tile + (all of it sees all keys)
  const uint16_t *list =
      p.mod.mask.ranges ? p.mod.mask.cols + ((long long)(rb % p.B) * n_qt + n) * n_qt : nullptr;
  const int m0 = p.causal ? n : 0;
  if (n_m == 0) {
    const bool part = p.kv_rep > 1;  // float per-rank partials
    const int per = part ? D / 4 : D / 8;
    for (int i = threadIdx.x; i < 128 * per; i += kThreads) {
      const int kvr = n * 128 + i / per, c = i % per;
      if (kvr >= p.S) break;
      const int s_rank = kvr / p.Sl, t = kvr - s_rank * p.Sl, rr = rb / p.B, bb = rb - rr * p.B;
      const size_t row = part ? ((size_t)hl_outer(p, rb, kvr) * p.Cs + kvr % p.Cs) * D
                              : (((size_t)(s_rank * p.B + bb) * p.Sl + t) * p.n_kv + (rr * p.kvp + kl)) * D;
      if (!in_range(p.status, (long long)row, D, p.dkv_n)) continue;
      const size_t es = part ? 4 : 2;
      *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(p.dk) + row * es + c * 16) = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(p.dv) + row * es + c * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int n_iter = p.group * n_m;
  // the query tile of step i
  auto tile_of = [&](int i) -> int {
    return list ? dev::col_at(p.mod.mask, list, i % n_m, p.status) >> 1 : m0 + i % n_m;
  };

  if (threadIdx.x == 0) {
    mbar_init(bar + kKBarIn, 1);
    for (int i = 0; i < kQSlots; ++i) {
      mbar_init(bar + kKBarQFull + 8 * i, 1);
      mbar_init(bar + kKBarQEmpty + 8 * i, 1);
    }
    for (int i = 0; i < kOSlots; ++i) {
      mbar_init(bar + kKBarOFull + 8 * i, 1);
      mbar_init(bar + kKBarOEmpty + 8 * i, 1);
    }
    mbar_init(bar + kKBarSFull, 1);
    mbar_init(bar + kKBarDPFull, 1);
    mbar_init(bar + kKBarPFull, 256);
    mbar_init(bar + kKBarDSFull, 256);
    mbar_init(bar + kKBarAcc, 1);
    mbar_init(bar + kKBarDrain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(bar + kKTmemSlot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::oBar + kKTmemSlot);
  const uint32_t tdV = tmem + 256, tdK = tmem + 256 + D;

  if (warp >= 8) {
    regs_dec<kRegsProducer>();
    if (warp == kTmaWarp) {
      if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmQ);
        mbar_arrive_expect_tx(bar + kKBarIn, 2 * L::kT);
        const int krow = n * 128 % p.Cs, ko = hl_outer(p, rb, n * 128);
        for (int c = 0; c < kCh; ++c) {
          tma_load_4d(sK + c * 16384, &tmK, bar + kKBarIn, c * 64, kl, krow, ko);
          tma_load_4d(sV + c * 16384, &tmV, bar + kKBarIn, c * 64, kl, krow, ko);
        }
        int issued_q = -1, issued_o = -1;
        for (int i = 0; i < n_iter; ++i) {
          const int qs = i % kQSlots, os = i % kOSlots;
          const int gi = i / n_m, m = tile_of(i), j = kl * p.group + gi;
          const int mrow = m * 128 % p.Cs, mo = hl_outer(p, rb, m * 128);
          if (!mbar_wait_bounded(bar + kKBarQEmpty + 8 * qs, ((i / kQSlots) & 1) ^ 1, abort_flag, gst)) break;
          mbar_arrive_expect_tx(bar + kKBarQFull + 8 * qs, L::kT + 512);
          for (int c = 0; c < kCh; ++c)
            tma_load_4d(sQ + qs * L::kT + c * 16384, &tmQ, bar + kKBarQFull + 8 * qs, c * 64, j, mrow, mo);
          dev::tma_load_2d(sDl + qs * 512, &tmDl, bar + kKBarQFull + 8 * qs, mrow, mo * p.hp + j);
          issued_q = i;
          if (!mbar_wait_bounded(bar + kKBarOEmpty + 8 * os, ((i / kOSlots) & 1) ^ 1, abort_flag, gst)) break;
          mbar_arrive_expect_tx(bar + kKBarOFull + 8 * os, L::kT + 512);
          for (int c = 0; c < kCh; ++c)
            tma_load_4d(sdO + os * L::kT + c * 16384, &tmdO, bar + kKBarOFull + 8 * os, c * 64, j, mrow, mo);
          dev::tma_load_2d(sL + os * 512, &tmL, bar + kKBarOFull + 8 * os, mrow, mo * p.hp + j);
          issued_o = i;
        }
        if (*abort_flag) {
          volatile int never = 0;
          mbar_wait_bounded(bar + kKBarIn, 0, &never, nullptr, 500000000ull);
          for (int i = issued_q - (kQSlots - 1); i <= issued_q; ++i)
            if (i >= 0)
              mbar_wait_bounded(bar + kKBarQFull + 8 * (i % kQSlots), (i / kQSlots) & 1, &never, nullptr,
                                500000000ull);
          for (int i = issued_o - (kOSlots - 1); i <= issued_o; ++i)
            if (i >= 0)
              mbar_wait_bounded(bar + kKBarOFull + 8 * (i % kOSlots), (i / kOSlots) & 1, &never, nullptr,
                                500000000ull);
        }
      }
    } else if (warp == kMmaWarp) {
      if (lane == 0) {
        constexpr uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);  // S^T, dP^T: both operands K-major
        constexpr uint32_t idA = idesc_bf16_f32(128, D, 0, 1);    // dV, dK: B (dO, Q) MN-major
        auto q_ready = [&](int i) -> bool {
          return mbar_wait_bounded(bar + kKBarQFull + 8 * (i % kQSlots), (i / kQSlots) & 1, abort_flag, gst);
        };
        auto o_ready = [&](int i) -> bool {
          return mbar_wait_bounded(bar + kKBarOFull + 8 * (i % kOSlots), (i / kOSlots) & 1, abort_flag, gst);
        };
        // S^T(i) = K Q_i^T (Q tile i has landed: the caller waited).
        auto issue_s = [&](int i) {
          const int qs = i % kQSlots;
          const uint64_t k = here(smem_desc_sw128(sK, 16, 1024)), q = here(smem_desc_sw128(sQ + qs * L::kT, 16, 1024));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            mma_bf16_ss(tmem, k + o, q + o, idS, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar + kKBarSFull);
        };
        // dP^T(i) = V dO_i^T (dO tile i has landed: the caller waited).
        auto issue_dp = [&](int i) {
          const int os = i % kOSlots;
          const uint64_t v = here(smem_desc_sw128(sV, 16, 1024)),
                         d = here(smem_desc_sw128(sdO + os * L::kT, 16, 1024));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            mma_bf16_ss(tmem + 128, v + o, d + o, idS, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar + kKBarDPFull);
        };
        // Q tile 1 as well: the burst dV(0) S^T(1) follows the P phase of step 0,
        // and later Q tiles are vouched for by the softmax's arrivals.
        bool ok = mbar_wait_bounded(bar + kKBarIn, 0, abort_flag, gst) && q_ready(0) && o_ready(0) &&
                  (n_iter < 2 || q_ready(1));
        if (ok && n_iter > 0) {
          tc_fence_after_sync();
          issue_s(0);
          issue_dp(0);
        }
        for (int i = 0; ok && i < n_iter; ++i) {
          const int qs = i % kQSlots, os = i % kOSlots;
          // burst 1: dV(i), S^T(i+1).  P^T / dS^T: queries 16kk..16kk+15 are
          // columns 8kk.. of warpgroup 0's half (kk < 4) or of warpgroup 1's
          // half at +64 (kk >= 4).
          if (!(ok = mbar_wait_bounded(bar + kKBarPFull, i & 1, abort_flag, gst))) break;
          tc_fence_after_sync();
          const uint64_t dO = here(smem_desc_sw128(sdO + os * L::kT, 16384, 1024));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t ac = (kk < 4 ? 0u : 64u) + (uint32_t)(kk & 3) * 8;
            mma_bf16_ts(tdV, tmem + ac, dO + (kk * 2048 >> 4), idA,
                        (i > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(bar + kKBarOEmpty + 8 * os);
          if (i + 1 < n_iter) issue_s(i + 1);
          // burst 2: dK(i), dP^T(i+1)
          if (!(ok = mbar_wait_bounded(bar + kKBarDSFull, i & 1, abort_flag, gst))) break;
          tc_fence_after_sync();
          const uint64_t q = here(smem_desc_sw128(sQ + qs * L::kT, 16384, 1024));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t ac = (kk < 4 ? 0u : 64u) + (uint32_t)(kk & 3) * 8;
            mma_bf16_ts(tdK, tmem + 128 + ac, q + (kk * 2048 >> 4), idA,
                        (i > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(bar + kKBarQEmpty + 8 * qs);
          if (i + 1 < n_iter) issue_dp(i + 1);
        }
        mma_commit(bar + kKBarAcc);
        mma_commit(bar + kKBarDrain);
        volatile int never = 0;
        mbar_wait_bounded(bar + kKBarDrain, 0, &never, nullptr);
      }
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ---------------------------------------------- softmax warpgroups
    const int g = warp >> 2, w4 = warp & 3;
    const int r = w4 * 32 + lane;  // key row within the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
    const int kvr = n * 128 + r;
    // dK's epilogue undoes the rotation of key row kvr: pairs [g*32, g*32+32)
    // (warpgroup 0 alone for D = 64)
    const bool rot = p.rope_cos && p.kv_rep == 1 && (D == 128 || g == 0) && kvr < p.S &&
                     in_range(p.status, (long long)kvr * (D / 2), D / 2, p.rope_n);
    const float *rcs = rot ? p.rope_cos + (size_t)kvr * (D / 2) + g * 32 : nullptr;
    const float *rsn = rot ? p.rope_sin + (size_t)kvr * (D / 2) + g * 32 : nullptr;
    if (rot) rope_prefetch(rcs, rsn);
    // The queries that see key kvr, [k_first, k_first + k_cnt); k_cnt -1: no
    // such interval, each query's interval of keys is looked up.
    int k_first = p.causal ? kvr : 0, k_cnt = max(p.S - k_first, 0);
    const long long row0 = (long long)(rb % p.B) * p.mod.mask.Sp;
    if (list) {
      const int2 kq = in_range(p.status, row0 + kvr, 1, p.mod.mask.rows_n) ? __ldg(p.mod.mask.keys + row0 + kvr)
                                                                           : make_int2(0, 0);
      k_first = kq.x, k_cnt = kq.y;
    }
    const bool odd = list && __any_sync(0xffffffffu, k_cnt < 0);
    // a bias is linear in what is seen where no query sees a key behind it
    const int side = __all_sync(0xffffffffu, k_cnt == 0 || (k_cnt > 0 && k_first >= kvr)) ? 1 : 0;
    int form = 0;  // the form of tanh this warp's tiles have needed so far
    bool ok = true;
    int i = 0;
    // Step i in form kForm, its scores masked by the thread's interval (kMask)
    // or not: false where it needs a further form, or (ok false) failed.
    auto step = [&](auto form_c, const auto &tools, auto mask_c, int q0, bool whole) -> bool {
      constexpr int kForm = decltype(form_c)::value;
      constexpr bool kMask = decltype(mask_c)::value;
      const int qs = i % kQSlots, os = i % kOSlots;
      if (!warp_wait(bar + kKBarSFull, i & 1, abort_flag, gst)) return ok = false;
      tc_fence_after_sync();
      uint32_t sr[2][32];
      tmem_ld32(tmem + lane_base + g * 64, sr[0]);
      tmem_ld32(tmem + lane_base + g * 64 + 32, sr[1]);
      // This step's LSE rides in its dO slot; after step 0 these threads
      // waited for that slot at the end of the previous step.
      if (i == 0 && !warp_wait(bar + kKBarOFull, 0, abort_flag, gst)) return ok = false;
      tmem_wait_ld();
      reg_fence(sr[0]);
      reg_fence(sr[1]);
      const int lo = k_first - q0;  // columns [lo, lo + k_cnt) of this warpgroup's 64 see the key
      const float2 *nl2 = reinterpret_cast<const float2 *>(smem + L::oL + os * 512) + g * 32;
      const float2 *dl2 = reinterpret_cast<const float2 *>(smem + L::oDl + qs * 512) + g * 32;
      float2 pf[32];  // P f of this thread's 64 columns, kept for dS
      uint32_t w[2][16];
      float slope2 = 0.f;
      if constexpr ((kMod & kModBias) != 0)
        slope2 = in_range(p.status, (rb / p.B) * p.hp + kl * p.group + i / n_m, 1, p.n_head)
                     ? __ldg(p.mod.slopes + (rb / p.B) * p.hp + kl * p.group + i / n_m) * kLog2e
                     : 0.f;
      const float big = p_mod<kMod, kForm, true, kMask>(
          sr, tools, p.scale_log2, slope2, q0 - kvr, side, [&](int c) { return dev::f2_of(nl2[c].x, nl2[c].y); }, lo,
          k_cnt, pf, w);
      if constexpr ((kMod & kModCap) != 0 && kForm < 2) {
        if (__any_sync(0xffffffffu, big > (kForm == 0 ? p.mod.lim2 : p.mod.lim4))) {
          form = dev::cap_form(big, p.mod);
          return false;  // (the scores are still in TMEM)
        }
      }
      if (odd && !whole) {  // each query's interval of keys
        const bool get = in_range(p.status, row0 + q0, 64, p.mod.mask.rows_n);
        const int4 *rg = reinterpret_cast<const int4 *>(p.mod.mask.ranges + row0 + q0);  // {lo, len} of two queries
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const int4 v = get ? __ldg(rg + c) : make_int4(0, 0, 0, 0);
          if ((unsigned)(kvr - v.x) >= (unsigned)v.y) pf[c].x = 0.f, w[c >> 4][c & 15] &= 0xffff0000u;
          if ((unsigned)(kvr - v.z) >= (unsigned)v.w) pf[c].y = 0.f, w[c >> 4][c & 15] &= 0x0000ffffu;
        }
      }
      tmem_st16(tmem + lane_base + g * 64, w[0]);
      tmem_st16(tmem + lane_base + g * 64 + 16, w[1]);
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(bar + kKBarPFull);

      if (!warp_wait(bar + kKBarDPFull, i & 1, abort_flag, gst)) return ok = false;
      // ... and its delta in its Q slot, which these threads waited for at the
      // end of step i-2 (steps 0 and 1: here).
      if (i < 2 && !warp_wait(bar + kKBarQFull + 8 * qs, 0, abort_flag, gst)) return ok = false;
      tc_fence_after_sync();
      uint32_t dr[2][32];
      tmem_ld32(tmem + lane_base + 128 + g * 64, dr[0]);
      tmem_ld32(tmem + lane_base + 128 + g * 64 + 32, dr[1]);
      tmem_wait_ld();
      reg_fence(dr[0]);
      reg_fence(dr[1]);
      ds_columns(dr, dl2, pf, w);
      tmem_st16(tmem + lane_base + 128 + g * 64, w[0]);
      tmem_st16(tmem + lane_base + 128 + g * 64 + 16, w[1]);
      tmem_wait_st();
      tc_fence_before_sync();
      // The issuer waits for this arrival alone before dK(i) dP^T(i+1) and
      // (as the last wait before it) dV(i+1) S^T(i+2), so it also vouches for
      // dO tile i+1 and Q tile i+2 having landed.  Waiting here, a step ahead
      // of S^T(i+2), keeps these waits off the softmax's P phase, which the
      // tensor core waits for.
      if (i + 1 < n_iter &&
          !warp_wait(bar + kKBarOFull + 8 * ((i + 1) % kOSlots), ((i + 1) / kOSlots) & 1, abort_flag, gst)) {
        return ok = false;
      }
      if (i + 2 < n_iter &&
          !warp_wait(bar + kKBarQFull + 8 * ((i + 2) % kQSlots), ((i + 2) / kQSlots) & 1, abort_flag, gst)) {
        return ok = false;
      }
      mbar_arrive(bar + kKBarDSFull);
      return true;
    };
    // The steps from i on in form kForm: false where step i needs a further one.
    auto run = [&](auto form_c) -> bool {
      const dev::CapFormSlope<(kMod & kModCap) ? decltype(form_c)::value : -1> tools(p.mod, dev::Nil());
#pragma unroll 1
      for (; i < n_iter; ++i) {
        int q0 = (m0 + i % n_m) * 128 + g * 64;
        bool whole = false;  // mask plan: nothing of the tile pair is masked
        if (list) {
          const int e = dev::col_at(p.mod.mask, list, i % n_m, p.status);
          q0 = (e >> 1) * 128 + g * 64;
          whole = e & 1;
        }
        const int lo = k_first - q0;
        const bool masked = !whole && !odd && !__all_sync(0xffffffffu, lo <= 0 && lo + k_cnt >= 64);
        if (!(masked ? step(form_c, tools, std::true_type{}, q0, whole)
                     : step(form_c, tools, std::false_type{}, q0, whole)))
          return !ok;
      }
      return true;
    };
    using std::integral_constant;
    if constexpr ((kMod & kModCap) == 0) {
      run(integral_constant<int, 0>{});
    } else {
      if (!run(integral_constant<int, 0>{}) && (form == 2 || !run(integral_constant<int, 1>{})))
        run(integral_constant<int, 2>{});
    }
    // ------------------------------------------------------------ epilogue
    RopeRow angles;
    if (ok && rot) rope_load(angles, rcs, rsn);
    if (ok) ok = warp_wait(bar + kKBarAcc, 0, abort_flag, gst);
    if (ok && p.kv_rep > 1) {
      // Replicated kv-head: this rank's q-heads give only part of dK, dV; the
      // raw fp32 accumulators go to the per-rank partial buffers and the sum
      // over the replicas (with scale and inverse rotation) follows.
      tc_fence_after_sync();
      const bool live = kvr < p.S;
      // partials [P*B][Cs][D]: the row of key kvr in this member's head layout
      const int kr = live ? kvr : 0;
      const size_t prow = (size_t)hl_outer(p, rb, kr) * p.Cs + kr % p.Cs;
      float *pv = reinterpret_cast<float *>(p.dv) + prow * D;
      float *pk = reinterpret_cast<float *>(p.dk) + prow * D;
      const bool put = live && in_range(p.status, (long long)(prow * D), D, p.dkv_n);
      // warpgroup g owns columns [g*D/2, (g+1)*D/2) of both accumulators; the
      // TMEM loads are warp-wide, only the stores depend on the row
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int col = g * (D / 2) + c * 32;
        uint32_t x[32], y[32];
        tmem_ld32(tdV + lane_base + col, x);
        tmem_ld32(tdK + lane_base + col, y);
        tmem_wait_ld();
        if (put) {
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            reinterpret_cast<uint4 *>(pv + col)[v] = make_uint4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
            reinterpret_cast<uint4 *>(pk + col)[v] = make_uint4(y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]);
          }
        }
      }
    } else if (ok) {
      tc_fence_after_sync();
      const bool live = kvr < p.S;
      const int s_rank = kvr / p.Sl, t = kvr - s_rank * p.Sl;
      const int rr = rb / p.B, bb = rb - rr * p.B;
      const size_t row = (((size_t)(s_rank * p.B + bb) * p.Sl + t) * p.n_kv + (rr * p.kvp + kl)) * D;
      const bool put = live && in_range(p.status, (long long)row, D, p.dkv_n) &&
                       (!p.rope_cos || in_range(p.status, (long long)kvr * (D / 2), D / 2, p.rope_n));
      // dV: warpgroup g owns columns [g*D/2, (g+1)*D/2)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[32];
        const int col = g * (D / 2) + c * 32;
        tmem_ld32(tdV + lane_base + col, x);
        tmem_wait_ld();
        if (put) store_plain(p.dv + row + col, x, 1.0f);
      }
      // dK: rotation pairs (i, i + D/2); warpgroup g owns i in [g*32, g*32+32)
      // for D = 128, warpgroup 0 owns all 32 pairs for D = 64.
      if (D == 128 || g == 0) {
        const int i0 = g * 32;
        uint32_t x[32], y[32];
        tmem_ld32(tdK + lane_base + i0, x);
        tmem_ld32(tdK + lane_base + D / 2 + i0, y);
        tmem_wait_ld();
        if (put) store_unrotated(p.dk + row + i0, p.dk + row + D / 2 + i0, x, y, p.scale, rot, angles);
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, (uint32_t)ULYSSES_STATUS_BWD_TIMEOUT);
}

// ================================================================== dQ kernel
// (TMEM and rings as in attn_bwd_tc.cu.)
constexpr int kKSlots = 3, kVSlots = 3;

enum : uint32_t {
  kQBarQReady = 0,                         // 256 arrivals: Q and dO are in TMEM
  kQBarKFull = 8,                          // [kKSlots]
  kQBarKEmpty = kQBarKFull + 8 * kKSlots,  // [kKSlots]
  kQBarVFull = kQBarKEmpty + 8 * kKSlots,  // [kVSlots]
  kQBarVEmpty = kQBarVFull + 8 * kVSlots,  // [kVSlots]
  kQBarSFull = kQBarVEmpty + 8 * kVSlots,
  kQBarSFree = kQBarSFull + 8,             // 256 arrivals
  kQBarDPFull = kQBarSFree + 8,
  kQBarDSFull = kQBarDPFull + 8,           // 256 arrivals
  kQBarAcc = kQBarDSFull + 8,
  kQBarTaken = kQBarAcc + 8,       // the answer on a block to take over is in kQTakenSlot
  kQBarItem = kQBarTaken + 8,      // [2] item n's facts are in slot n & 1 of kQItemSlot
  kQBarItemEmpty = kQBarItem + 16, // [2] every warp is through with that item
  kQBarDrain = kQBarItemEmpty + 16,
  kQTmemSlot = kQBarDrain + 8,
  kQAbortSlot = kQTmemSlot + 4,
  kQTakenSlot = (kQAbortSlot + 4 + 15) / 16 * 16,
  kQItemSlot = kQTakenSlot + 16  // [2] x 32 bytes
};
constexpr int kAhead = 3;  // key tiles before its end at which an item's successor is asked for
static_assert(kQItemSlot + 64 <= 512, "dQ barrier block");

template <int D>
struct QLayout {
  static constexpr uint32_t kT = 128u * D * 2;  // one 128-row tile of K or V
  static constexpr uint32_t oK = 0, oV = kKSlots * kT, oBar = oV + kVSlots * kT;
  static constexpr uint32_t kAlloc = oBar + 512 + 1024;
};

// dS = P * (dP - delta) for the same 64 columns, packed to bf16.
__device__ __forceinline__ void ds_row(const uint32_t (&d)[2][32], const float2 (&pf)[32], float dlt,
                                       uint32_t (&w)[2][16]) {
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const uint32_t *dh = d[c >> 4];
    const int e = 2 * (c & 15);
    const float2 y = sub2(make_float2(__uint_as_float(dh[e]), __uint_as_float(dh[e + 1])), make_float2(dlt, dlt));
    const float2 ds = mul2(pf[c], y);
    w[c >> 4][c & 15] = pack_bf16x2(ds.x, ds.y);
  }
}

// The item of a block: one query tile of a head, key tiles [t0, t0 + nB) (nA:
// its CTA's items with keys before).
__device__ __forceinline__ Item dq_item(const BwdParams &p, int block) {
  const int n_qt = (p.S + 127) / 128;
  const dev::HeadTile ht = dev::grouped_order(block, p.Pu * p.B * p.hp, n_qt, p.group_q);
  Item it;
  it.tile = n_qt - 1 - ht.rank;  // longest tiles first
  it.j = ht.head % p.hp;
  it.rb = ht.head / p.hp;
  it.t0 = it.nA = 0;
  it.nB = p.causal ? min(n_qt, it.tile + 1) : n_qt;
  if (p.mod.mask.ranges) {
    const int4 tl = dev::tile_at(p.mod.mask, (long long)(it.rb % p.B) * n_qt + it.tile, p.status);
    it.t0 = tl.x / 128;
    it.nB = max((tl.y + 127) / 128 - it.t0, 0);
  }
  return it;
}

template <int D, int kMod>
__global__ void __launch_bounds__(kThreads, 1)
    dq_mod_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                  const BwdParams p) {
  using L = QLayout<D>;
  constexpr int kCh = D / 64;
  constexpr uint32_t kColDP = 128, kColDQ = 256, kColQ = 384, kColDO = 448;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t *smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const uint32_t sK = sb + L::oK, sV = sb + L::oV, bar = sb + L::oBar;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::oBar + kQAbortSlot);
  const volatile uint32_t *gst = p.status;
  const Checks checks(p);
  const Item first = dq_item(p, (int)blockIdx.x);
  if (!checks.fine(p)) return;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar + kQBarQReady, 256);
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(bar + kQBarKFull + 8 * i, 1);
      mbar_init(bar + kQBarKEmpty + 8 * i, 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(bar + kQBarVFull + 8 * i, 1);
      mbar_init(bar + kQBarVEmpty + 8 * i, 1);
    }
    mbar_init(bar + kQBarSFull, 1);
    mbar_init(bar + kQBarSFree, 256);
    mbar_init(bar + kQBarDPFull, 1);
    mbar_init(bar + kQBarDSFull, 256);
    mbar_init(bar + kQBarAcc, 1);
    mbar_init(bar + kQBarTaken, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + kQBarItem + 8 * i, 1);
      mbar_init(bar + kQBarItemEmpty + 8 * i, 9);  // the softmax warps and the issuer
    }
    put_item(bar + kQItemSlot, first);
    mbar_init(bar + kQBarDrain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(bar + kQTmemSlot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::oBar + kQTmemSlot);
  const uint32_t tdQ = tmem + kColDQ;
  // The facts of this CTA's n-th item (from the second on, once kQBarItem says so).
  auto item_slot = [&](int n) { return bar + kQItemSlot + 32 * (n & 1); };
  auto item_parity = [](int n) { return (uint32_t)(((n - 1) >> 1) & 1); };

  if (warp >= 8) {
    regs_dec<kRegsProducer>();
    if (warp == kTmaWarp) {
      if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        int issued_k = -1, issued_v = -1;  // the last ring entries filled
        bool ok = true;
        Item it = get_item(item_slot(0)), next;
        // Takes over a block that has not started as the n-th item (n >= 1) and asks
        // L2 for the rows that it reads first.  (The answer is waited for in any
        // case: it lands in this CTA's shared memory.)
        auto take = [&](int n) -> bool {
          if (n > 1 && !mbar_wait_bounded(bar + kQBarItemEmpty + 8 * (n & 1), ((n - 2) >> 1) & 1, abort_flag, gst))
            return false;
          mbar_arrive_expect_tx(bar + kQBarTaken, 16);
          dev::take_block(bar + kQTakenSlot, bar + kQBarTaken);
          volatile int never = 0;
          if (!mbar_wait_bounded(bar + kQBarTaken, (n - 1) & 1, &never, nullptr)) {
            *abort_flag = 1;
            return false;
          }
          const int block = dev::taken_block(bar + kQTakenSlot);
          if (block >= 0) {
            next = dq_item(p, block);
            next.nA = it.nA + (it.nB > 0 ? 1 : 0);
          } else {
            next.tile = -1;
          }
          put_item(item_slot(n), next);
          mbar_arrive(bar + kQBarItem + 8 * (n & 1));
          if (block >= 0 && next.nB > 0) {
            const int row = next.tile * 128 % p.Cs, outer = hl_outer(p, next.rb, next.tile * 128);
            for (int c = 0; c < kCh; ++c) {
              tma_prefetch_4d(&tmQ, c * 64, next.j, row, outer);
              tma_prefetch_4d(&tmdO, c * 64, next.j, row, outer);
            }
          }
          return true;
        };
        for (int n = 0;; ++n) {
          const int kl = it.j / p.group;
          for (int i = 0; i < it.nB; ++i) {
            const int e = issued_v + 1, ks = e % kKSlots, vs = e % kVSlots;
            if (!(ok = mbar_wait_bounded(bar + kQBarKEmpty + 8 * ks, ((e / kKSlots) & 1) ^ 1, abort_flag, gst))) break;
            mbar_arrive_expect_tx(bar + kQBarKFull + 8 * ks, L::kT);
            const int krow = (it.t0 + i) * 128 % p.Cs, ko = hl_outer(p, it.rb, (it.t0 + i) * 128);
            for (int c = 0; c < kCh; ++c)
              tma_load_4d(sK + ks * L::kT + c * 16384, &tmK, bar + kQBarKFull + 8 * ks, c * 64, kl, krow, ko);
            issued_k = e;
            if (!(ok = mbar_wait_bounded(bar + kQBarVEmpty + 8 * vs, ((e / kVSlots) & 1) ^ 1, abort_flag, gst))) break;
            mbar_arrive_expect_tx(bar + kQBarVFull + 8 * vs, L::kT);
            for (int c = 0; c < kCh; ++c)
              tma_load_4d(sV + vs * L::kT + c * 16384, &tmV, bar + kQBarVFull + 8 * vs, c * 64, kl, krow, ko);
            issued_v = e;
            if (i == max(it.nB - kAhead, 0) && !(ok = take(n + 1))) break;
          }
          if (!ok || (it.nB == 0 && !take(n + 1)) || next.tile < 0) break;
          it = next;
        }
        if (*abort_flag) {
          volatile int never = 0;
          for (int i = issued_k - (kKSlots - 1); i <= issued_k; ++i)
            if (i >= 0)
              mbar_wait_bounded(bar + kQBarKFull + 8 * (i % kKSlots), (i / kKSlots) & 1, &never, nullptr,
                                500000000ull);
          for (int i = issued_v - (kVSlots - 1); i <= issued_v; ++i)
            if (i >= 0)
              mbar_wait_bounded(bar + kQBarVFull + 8 * (i % kVSlots), (i / kVSlots) & 1, &never, nullptr,
                                500000000ull);
        }
      }
    } else if (warp == kMmaWarp) {
      if (lane == 0) {
        constexpr uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);  // S, dP: A (TMEM) and K, V K-major
        constexpr uint32_t idQ = idesc_bf16_f32(128, D, 0, 1);    // dQ: B (K tile) MN-major
        auto k_ready = [&](int i) -> bool {
          return mbar_wait_bounded(bar + kQBarKFull + 8 * (i % kKSlots), (i / kKSlots) & 1, abort_flag, gst);
        };
        auto v_ready = [&](int i) -> bool {
          return mbar_wait_bounded(bar + kQBarVFull + 8 * (i % kVSlots), (i / kVSlots) & 1, abort_flag, gst);
        };
        // S_i = Q K_i^T (Q: D elements 16kk.. are TMEM columns kColQ + 8kk ..);
        // K_i has landed (the caller waited).
        auto issue_s = [&](int i) {
          const int ks = i % kKSlots;
          const uint64_t k = here(smem_desc_sw128(sK + ks * L::kT, 16, 1024));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ts(tmem, tmem + kColQ + kk * 8, k + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), idS,
                        kk > 0 ? 1u : 0u);
          mma_commit(bar + kQBarSFull);
        };
        // dP_i = dO V_i^T (V_i has landed: the caller waited).
        auto issue_dp = [&](int i) {
          const int vs = i % kVSlots;
          const uint64_t v = here(smem_desc_sw128(sV + vs * L::kT, 16, 1024));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ts(tmem + kColDP, tmem + kColDO + kk * 8, v + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), idS,
                        kk > 0 ? 1u : 0u);
          mma_commit(bar + kQBarDPFull);
          mma_commit(bar + kQBarVEmpty + 8 * vs);
        };
        // One wait per burst (a thread with MMAs in flight stalls on its next
        // shared-memory access): the softmax's SFree and DSFull arrivals also
        // vouch for K tile i+1 and V tile i+1.
        // (Ring entries, S, dP and dS are counted through all items: i0 is the
        // item's first.)
        bool ok = true;
        int i0 = 0, n_live = 0;
        Item it = get_item(item_slot(0));
        for (int n = 0; it.tile >= 0; ++n) {
          const int end = i0 + it.nB;
          if (it.nB > 0) {
            if (!(ok = mbar_wait_bounded(bar + kQBarQReady, n_live & 1, abort_flag, gst) && k_ready(i0) && v_ready(i0)))
              break;
            ++n_live;
            tc_fence_after_sync();
            issue_s(i0);
            issue_dp(i0);
          }
          for (int i = i0; i < end; ++i) {
            // burst 1: S_{i+1}, once the softmax has loaded S_i
            if (i + 1 < end) {
              if (!(ok = mbar_wait_bounded(bar + kQBarSFree, i & 1, abort_flag, gst))) break;
              tc_fence_after_sync();
              issue_s(i + 1);
            }
            // burst 2: dQ += dS_i K_i, dP_{i+1}.  Keys 16kk.. of dS_i are columns
            // 8kk.. of warpgroup 0's half (kk < 4) or of warpgroup 1's half at +64.
            if (!(ok = mbar_wait_bounded(bar + kQBarDSFull, i & 1, abort_flag, gst))) break;
            tc_fence_after_sync();
            const int ks = i % kKSlots;
            const uint64_t k = here(smem_desc_sw128(sK + ks * L::kT, 16384, 1024));
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t ac = kColDP + (kk < 4 ? 0u : 64u) + (uint32_t)(kk & 3) * 8;
              mma_bf16_ts(tdQ, tmem + ac, k + (kk * 2048 >> 4), idQ,
                          (i > i0 || kk > 0) ? 1u : 0u);
            }
            mma_commit(bar + kQBarKEmpty + 8 * ks);
            if (i + 1 < end) issue_dp(i + 1);
          }
          if (!ok) break;
          if (it.nB > 0) mma_commit(bar + kQBarAcc);
          i0 = end;
          mbar_arrive(bar + kQBarItemEmpty + 8 * (n & 1));
          if (!(ok = mbar_wait_bounded(bar + kQBarItem + 8 * ((n + 1) & 1), item_parity(n + 1), abort_flag, gst)))
            break;
          it = get_item(item_slot(n + 1));
        }
        mma_commit(bar + kQBarDrain);
        volatile int never = 0;
        mbar_wait_bounded(bar + kQBarDrain, 0, &never, nullptr);
      }
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ---------------------------------------- softmax warpgroups: warpgroup g
    // owns key columns [64g, 64g+64) of every tile.
    const int g = warp >> 2, w4 = warp & 3;
    const int r = w4 * 32 + lane;  // query row within the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
    constexpr bool kBias = (kMod & kModBias) != 0;
    // What an item's row needs from global memory beside its tiles: its factors
    // (nlse, delta) and the keys it sees, {first, how many}.
    // (As of an empty row until an item with keys comes.)
    float nl2 = 0.f, dlt = 0.f;
    int2 keys = make_int2(0, 0);
    // Starts an item: brings these, and (warpgroup 0) this thread's Q row or
    // (warpgroup 1) its dO row, into TMEM (rows past S are zero).  The item
    // before has formed its last S and dP.
    auto load_rows = [&](const Item &it) {
      const int qi = it.tile * 128 + r, qr = qi < p.S ? qi : 0;
      const size_t hl = (size_t)hl_outer(p, it.rb, qr);
      const size_t qoff = ((hl * p.Cs + qr % p.Cs) * p.hp + it.j) * D;
      const __nv_bfloat16 *src = (g == 0 ? p.q : p.dout) + qoff;
      const bool get = qi < p.S && in_range(p.status, (long long)qoff, D, p.qo_n);
      uint32_t x[D / 64][32];
      if (!get) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) x[c][e] = 0u;
      } else if (p.qo_by32) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int v = 0; v < 4; ++v) ld_global_32(&x[c][8 * v], src + c * 64 + v * 16);
      } else {
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src) + c * 8 + v);
            x[c][4 * v] = u.x;
            x[c][4 * v + 1] = u.y;
            x[c][4 * v + 2] = u.z;
            x[c][4 * v + 3] = u.w;
          }
      }
      const size_t lrow = (hl * p.hp + it.j) * p.Ld + qr % p.Cs;
      const bool get_row = qi < p.S && in_range(p.status, (long long)lrow, 1, p.rows_n);
      nl2 = get_row ? p.nlse[lrow] : 0.f;
      dlt = get_row ? p.delta[lrow] : 0.f;
      keys = make_int2(0, p.causal ? min(qi + 1, p.S) : p.S);
      if (p.mod.mask.ranges) {
        const long long ri = (long long)(it.rb % p.B) * p.mod.mask.Sp + qi;
        keys = in_range(p.status, ri, 1, p.mod.mask.rows_n) ? __ldg(p.mod.mask.ranges + ri) : make_int2(0, 0);
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) tmem_st32(tmem + lane_base + (g == 0 ? kColQ : kColDO) + c * 32, x[c]);
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(bar + kQBarQReady);
    };
    if (first.nB > 0) load_rows(first);
    bool ok = true;
    // dQ's epilogue undoes the rotation of query row qi: pairs [g*32, g*32+32)
    // (warpgroup 0 alone for D = 64)
    auto turns = [&](int qi) {
      return p.rope_cos && (D == 128 || g == 0) && qi < p.S &&
             in_range(p.status, (long long)qi * (D / 2), D / 2, p.rope_n);
    };
    int i = 0;  // the key tile's ring entry, counted through all items
#pragma unroll 1
    for (int n = 0;; ++n) {
      int end, koff;  // of the item's tiles; of key tile i: 128 i + koff is this warpgroup's first key
      int qi;
      float slope2 = 0.f, zero;
      {
        const Item it = get_item(item_slot(n));
        end = i + it.nB, koff = (it.t0 - i) * 128 + g * 64, qi = it.tile * 128 + r, zero = it.zero;
        if constexpr (kBias) slope2 = dev::slope_at(p.mod, (it.rb / p.B) * p.hp + it.j, p.n_head, p.status);
        if (turns(qi))
          rope_prefetch(p.rope_cos + (size_t)qi * (D / 2) + g * 32, p.rope_sin + (size_t)qi * (D / 2) + g * 32);
      }
      // The keys this row sees, [k_lo, k_hi): all of them where it sees none (its
      // nlse is -inf, so P = 0: no masking).
      const bool dead = keys.y == 0;
      const int k_lo = dead ? -(1 << 29) : keys.x, k_hi = dead ? 1 << 29 : keys.x + keys.y;
      // a bias is linear in what is seen where no row sees a key ahead of it
      const int side = __all_sync(0xffffffffu, dead || qi >= p.S || k_hi <= qi + 1) ? -1 : 0;
      int form = 0;  // the form of tanh this warp's tiles have needed so far
      // As in the dK/dV kernel.
      auto step = [&](auto form_c, const auto &tools, auto mask_c, int k0) -> bool {
        constexpr int kForm = decltype(form_c)::value;
        constexpr bool kMask = decltype(mask_c)::value;
        if (!warp_wait(bar + kQBarSFull, i & 1, abort_flag, gst)) return ok = false;
        tc_fence_after_sync();
        uint32_t sr[2][32];
        tmem_ld32(tmem + lane_base + g * 64, sr[0]);
        tmem_ld32(tmem + lane_base + g * 64 + 32, sr[1]);
        tmem_wait_ld();
        reg_fence(sr[0]);
        reg_fence(sr[1]);
        if constexpr ((kMod & kModCap) != 0 && kForm < 2) {
          const float big = dev::largest_square(sr);
          if (__any_sync(0xffffffffu, big > (kForm == 0 ? p.mod.lim2 : p.mod.lim4))) {
            form = dev::cap_form(big, p.mod);
            return false;  // (the scores are still in TMEM)
          }
        }
        tc_fence_before_sync();
        // The issuer waits for this arrival alone before S_{i+1}, so it also
        // vouches for K tile i+1 having landed.
        if (i + 1 < end &&
            !warp_wait(bar + kQBarKFull + 8 * ((i + 1) % kKSlots), ((i + 1) / kKSlots) & 1, abort_flag, gst)) {
          return ok = false;
        }
        mbar_arrive(bar + kQBarSFree);
        float2 pf[32];
        const dev::f2x off = dev::f2_of(nl2, nl2);
        uint32_t wd[2][16];
        p_mod<kMod, kForm, false, kMask>(sr, tools, p.scale_log2, slope2, k0 - qi, side, [&](int) { return off; },
                                         k_lo - k0, k_hi - k_lo, pf, wd);
        if (!warp_wait(bar + kQBarDPFull, i & 1, abort_flag, gst)) return ok = false;
        tc_fence_after_sync();
        uint32_t dr[2][32];
        tmem_ld32(tmem + lane_base + kColDP + g * 64, dr[0]);
        tmem_ld32(tmem + lane_base + kColDP + g * 64 + 32, dr[1]);
        tmem_wait_ld();
        reg_fence(dr[0]);
        reg_fence(dr[1]);
        ds_row(dr, pf, dlt, wd);
        tmem_st16(tmem + lane_base + kColDP + g * 64, wd[0]);
        tmem_st16(tmem + lane_base + kColDP + g * 64 + 16, wd[1]);
        tmem_wait_st();
        tc_fence_before_sync();
        // ... and this one alone before dQ(i) and dP_{i+1}: V tile i+1 too.
        if (i + 1 < end &&
            !warp_wait(bar + kQBarVFull + 8 * ((i + 1) % kVSlots), ((i + 1) / kVSlots) & 1, abort_flag, gst)) {
          return ok = false;
        }
        mbar_arrive(bar + kQBarDSFull);
        return true;
      };
      auto run = [&](auto form_c) -> bool {
        const dev::CapFormSlope<(kMod & kModCap) ? decltype(form_c)::value : -1> tools(p.mod, zero);
#pragma unroll 1
        for (; i < end; ++i) {
          const int k0 = i * 128 + koff;
          // columns [k_lo - k0, k_hi - k0) of this warpgroup's 64 are seen
          const bool masked = !__all_sync(0xffffffffu, k_lo - k0 <= 0 && k_hi - k0 >= 64);
          if (!(masked ? step(form_c, tools, std::true_type{}, k0) : step(form_c, tools, std::false_type{}, k0)))
            return !ok;
        }
        return true;
      };
      using std::integral_constant;
      if constexpr ((kMod & kModCap) == 0) {
        run(integral_constant<int, 0>{});
      } else {
        if (!run(integral_constant<int, 0>{}) && (form == 2 || !run(integral_constant<int, 1>{})))
          run(integral_constant<int, 2>{});
      }
      // The next item's rows go to TMEM while this one's last products are formed.
      bool more = false;
      if (ok) ok = warp_wait(bar + kQBarItem + 8 * ((n + 1) & 1), item_parity(n + 1), abort_flag, gst);
      if (ok) {
        const Item next = get_item(item_slot(n + 1));
        more = next.tile >= 0;
        if (more && next.nB > 0) load_rows(next);
      }
      const Item it = get_item(item_slot(n));
      qi = it.tile * 128 + r;
      const int s_rank = qi / p.Sl, rr = it.rb / p.B;
      const size_t row =
          (((size_t)(s_rank * p.B + it.rb - rr * p.B) * p.Sl + qi - s_rank * p.Sl) * p.n_head + (rr * p.hp + it.j)) * D;
      const bool store = qi < p.S && in_range(p.status, (long long)row, D, p.dq_n) &&
                         (!p.rope_cos || in_range(p.status, (long long)qi * (D / 2), D / 2, p.rope_n));
      if (it.nB == 0) {  // no row sees a key
        for (int c = g * (D / 2); ok && store && c < (g + 1) * (D / 2); c += 8)
          *reinterpret_cast<uint4 *>(p.dq + row + c) = make_uint4(0u, 0u, 0u, 0u);
      } else if (ok) {
        const bool rot = turns(qi);
        const float *cs = p.rope_cos + (size_t)qi * (D / 2) + g * 32, *sn = p.rope_sin + (size_t)qi * (D / 2) + g * 32;
        RopeHalf angles;
        if (rot) rope_load(angles, cs, sn);
        ok = warp_wait(bar + kQBarAcc, it.nA & 1, abort_flag, gst);
        if (ok && (D == 128 || g == 0)) {
          tc_fence_after_sync();
#pragma unroll 1
          for (int c0 = 0; c0 < 32; c0 += 16) {
            uint32_t x[16], y[16];
            dev::tmem_ld16(tdQ + lane_base + g * 32 + c0, x);
            dev::tmem_ld16(tdQ + lane_base + D / 2 + g * 32 + c0, y);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(x[e]), "+r"(y[e]));  // no use before the wait
            __nv_bfloat16 *dst = p.dq + row + g * 32 + c0;
            if (store) store_unrotated(dst, dst + D / 2, x, y, p.scale, rot, angles, p.dq_by32);
            if (rot && c0 == 0) rope_load(angles, cs + 16, sn + 16);
          }
        }
      }
      if (!ok || !more) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + kQBarItemEmpty + 8 * (n & 1));
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, (uint32_t)ULYSSES_STATUS_BWD_TIMEOUT);
}

template <int D, int kMod>
cudaError_t launch_as(const BwdParams &bp, const CUtensorMap &mK, const CUtensorMap &mV, const CUtensorMap &mQ,
                      const CUtensorMap &mdO, const CUtensorMap &mL, const CUtensorMap &mDl, unsigned kv_blocks,
                      unsigned q_blocks, cudaStream_t st) {
  const auto dkdv = dkdv_mod_kernel<D, kMod>;
  const auto dq = dq_mod_kernel<D, kMod>;
  cudaError_t e = cudaFuncSetAttribute(dkdv, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)KVLayout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  dkdv<<<kv_blocks, kThreads, KVLayout<D>::kAlloc, st>>>(mK, mV, mQ, mdO, mL, mDl, bp);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)QLayout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  dq<<<q_blocks, kThreads, QLayout<D>::kAlloc, st>>>(mK, mV, mQ, mdO, bp);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const ulysses_problem &p, const TmaEncoder &enc, const void *q, const void *k, const void *v,
                     const void *do_head, const float *nlse, const float *delta, const void *ws, void *dq, void *dk,
                     void *dv, uint32_t *status, const ulysses_score_mod &m, cudaStream_t st) {
  const int Pu = group_ranks(p), Cs = chunk_len(p);
  const int hp = p.n_head / Pu, kvp = kv_per_rank(p), PB = p.P * p.B, UB = Pu * p.B;
  CUtensorMap mK, mV, mQ, mdO, mL, mDl;  // [P*B][Cs][hp|kvp][D]; the delta / nlse rows [P*B*hp][Cs] (Ld apart)
  if (!make_act_map(enc, &mK, k, D, kvp, Cs, PB, 128) || !make_act_map(enc, &mV, v, D, kvp, Cs, PB, 128) ||
      !make_act_map(enc, &mQ, q, D, hp, Cs, PB, 128) || !make_act_map(enc, &mdO, do_head, D, hp, Cs, PB, 128) ||
      !make_row_map(enc, &mL, nlse, Cs, delta_ld(p), PB * hp, 128) ||
      !make_row_map(enc, &mDl, delta, Cs, delta_ld(p), PB * hp, 128))
    return cudaErrorInvalidValue;
  BwdParams bp;
  bp.B = p.B;
  bp.S = p.S;
  bp.Sl = p.S / p.P;
  bp.hp = hp;
  bp.kvp = kvp;
  bp.group = hp / kvp;
  bp.causal = p.causal;
  bp.n_head = p.n_head;
  bp.n_kv = p.n_kv_head;
  bp.Pu = Pu;
  bp.Cs = Cs;
  bp.Ld = delta_ld(p);
  bp.dq_n = bp.qo_n = (long long)p.B * p.S * p.n_head * D;
  bp.dkv_n = kv_replicas(p) > 1 ? (long long)p.P * p.B * Cs * D : (long long)p.B * p.S * p.n_kv_head * D;
  bp.rows_n = (long long)PB * hp * bp.Ld;
  bp.rope_n = (long long)p.S * (D / 2);
  // CTA units: (group member, batch, head), each over the full sequence; the
  // plain backward's groups (their tiles stay in L2).
  const long long n_t = (p.S + 127) / 128, n_kv = (long long)UB * kvp, n_q = n_kv * bp.group;
  if (n_t * n_kv > 0x7fffffffll || n_t * n_q > 0x7fffffffll) return cudaErrorInvalidValue;
  bp.group_kv = l2_head_group((size_t)4 * p.S * D * bp.group, (int)n_kv, n_t * n_kv, (size_t)32 << 20);
  bp.group_q = l2_head_group((size_t)4 * p.S * D / bp.group, (int)n_q, n_t * n_q, (size_t)16 << 20);
  bp.scale = p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf((float)D);
  bp.scale_log2 = bp.scale * kLog2e;
  bp.nlse = nlse;
  bp.delta = delta;
  bp.q = static_cast<const __nv_bfloat16 *>(q);
  bp.dout = static_cast<const __nv_bfloat16 *>(do_head);
  bp.rope_cos = bp.rope_sin = nullptr;
  if (p.use_rope) {
    bp.rope_cos = reinterpret_cast<const float *>(static_cast<const uint8_t *>(ws) + workspace_layout(p).rope);
    bp.rope_sin = bp.rope_cos + (size_t)p.S * (D / 2);
  }
  bp.dq_by32 = (reinterpret_cast<uintptr_t>(dq) & 31) == 0;
  bp.qo_by32 = ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(do_head)) & 31) == 0;
  bp.kv_rep = kv_replicas(p);
  bp.dq = static_cast<__nv_bfloat16 *>(dq);
  bp.dk = static_cast<__nv_bfloat16 *>(dk);
  bp.dv = static_cast<__nv_bfloat16 *>(dv);
  bp.status = status;
  bp.rope_key = rope_key(p);
  bp.mod = score_mod(p, m);
  const unsigned kb = (unsigned)(n_t * n_kv), qb = (unsigned)(n_t * n_q);
  switch (score_mod_flags(m)) {
    case kModOn: return launch_as<D, kModOn>(bp, mK, mV, mQ, mdO, mL, mDl, kb, qb, st);
    case kModOn | kModCap: return launch_as<D, kModOn | kModCap>(bp, mK, mV, mQ, mdO, mL, mDl, kb, qb, st);
    case kModOn | kModBias: return launch_as<D, kModOn | kModBias>(bp, mK, mV, mQ, mdO, mL, mDl, kb, qb, st);
    case kModOn | kModCap | kModBias:
      return launch_as<D, kModOn | kModCap | kModBias>(bp, mK, mV, mQ, mdO, mL, mDl, kb, qb, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_attn_bwd_mod(const ulysses_problem &p, const TmaEncoder &enc, const void *q, const void *k,
                                const void *v, const void *do_head, const float *nlse, const float *delta,
                                const void *ws, void *dq_seq, void *dk, void *dv, uint32_t *status,
                                const ulysses_score_mod &mod, cudaStream_t st) {
  if (p.head_dim == 128)
    return launch_d<128>(p, enc, q, k, v, do_head, nlse, delta, ws, dq_seq, dk, dv, status, mod, st);
  if (p.head_dim == 64)
    return launch_d<64>(p, enc, q, k, v, do_head, nlse, delta, ws, dq_seq, dk, dv, status, mod, st);
  return cudaErrorInvalidValue;
}

}  // namespace ulysses
