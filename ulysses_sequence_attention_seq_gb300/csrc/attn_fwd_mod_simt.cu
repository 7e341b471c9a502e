// attn_fwd_mod_simt.cu -- fp32 attention forward with modified scores, on the
// CUDA cores.
//
// O_i = sum_k P_ik v_k with the scores of score_mod.cuh, in float throughout
// (the plain fp32 forward's reason: 1e-4 agreement, which rounded operands on
// the tensor cores do not give).  FMA throughput is the bound: 4 D per pair
// against 80 TFLOP/s.
//
// A block owns 32 query rows of one head and its kWarps warps split the keys:
// warp w takes the key tiles w, w + kWarps, ... of the rows' hull with its own
// running maximum and sum, and the warps' results are joined at the end, so
// short sequences still fill the chip and no warp waits for another meanwhile.
// A warp computes a 32 x kKeys tile: lane (tq, tk) = (lane / 4, lane % 4) holds
// rows tq + 8 i of S for keys tk + 4 j and, of O, the dimensions 16 j + 4 tk ..
// + 3.  Products are packed pairs: S pairs neighbouring dimensions (even and
// odd partial sums, added at the end), O neighbouring dimensions.  Q, K and P
// rows are padded by 16 bytes, so the 8 (or 4) rows a load touches lie in
// different banks.  K of the next tile is fetched while P V runs and V while
// the scores are formed.
// 1000 tokens, 8 heads of 64, all pairs: 64 us, 32 TFLOP/s (one thread per row:
// 414 us; 16-key tiles 72 us, eight warps a block 66 us).
#include <math.h>
#include <stdint.h>

#include "check.cuh"
#include "internal.h"
#include "score_mod.cuh"
#include "sm100.cuh"

namespace ulysses {
namespace {

using namespace sm100;

constexpr int kRows = 32, kWarps = 4;

template <int D>
struct Tile {
  static constexpr int kKeys = D == 128 ? 16 : 32;
  static constexpr int ldQ = D + 4, ldK = D + 4, ldP = kKeys + 4;
  static constexpr int kK = kKeys * ldK, kV = kKeys * D, kP = kRows * ldP;
  // K, V and P of a warp; at the end its 32 rows of O lie over K and V
  static constexpr int kWarpFloats = (kK + kV > kRows * D ? kK + kV : kRows * D) + kP;
  static constexpr int kQ = kRows * ldQ;
  static constexpr size_t kBytes = 4 * (size_t)(kQ + kWarps * kWarpFloats + 2 * kWarps * kRows);
};

struct SimtParams {
  const float *q, *k, *v;
  float *o, *lse;
  int S, B, n_head, hp, kvp, group, causal;
  float scale_log2;
  uint32_t *status;
  long long qo_n, kv_n, lse_n;
  dev::ScoreMod mod;
};

__device__ __forceinline__ void cp16(void *dst, const float *src, bool get) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(get ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) attn_fwd_mod_simt_kernel(const SimtParams p) {
  using T = Tile<D>;
  constexpr int kKeys = T::kKeys, nJ = kKeys / 4, nD = D / 16;
  extern __shared__ __align__(16) float smem[];
  if (!dev::mask_matches(p.mod.mask)) {
    if (threadIdx.x == 0) atomicOr(p.status, (uint32_t)ULYSSES_STATUS_MASK);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tq = lane >> 2, tk = lane & 3;
  const int n_qt = (p.S + kRows - 1) / kRows;
  const int q0 = (n_qt - 1 - (int)(blockIdx.x % n_qt)) * kRows;  // long causal rows first
  const long long hid = blockIdx.x / n_qt;                       // (r*B + b)*hp + j
  const int j = (int)(hid % p.hp);
  const long long rb = hid / p.hp;
  const int b = (int)(rb % p.B);
  const long long q_base = (rb * p.S * p.hp + j) * D, kv_base = (rb * p.S * p.kvp + j / p.group) * D;
  float *sQ = smem, *mine = smem + T::kQ + warp * T::kWarpFloats;
  float *sK = mine, *sV = mine + T::kK, *sP = mine + T::kWarpFloats - T::kP;
  float *sM = smem + T::kQ + kWarps * T::kWarpFloats, *sL = sM + kWarps * kRows;

  // lane i finds what row q0 + i sees; the warp takes the hull
  int r_lo = 0, r_hi = 0;
  if (q0 + lane < p.S) {
    if (p.mod.mask.ranges) {
      const long long ri = (long long)b * p.mod.mask.Sp + q0 + lane;
      const int2 rg = in_range(p.status, ri, 1, p.mod.mask.rows_n) ? __ldg(p.mod.mask.ranges + ri) : make_int2(0, 0);
      r_lo = rg.x, r_hi = rg.x + rg.y;
    } else {
      r_hi = p.causal ? q0 + lane + 1 : p.S;
    }
  }
  int h_lo = r_hi > r_lo ? r_lo : INT_MAX, h_hi = r_hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    h_lo = min(h_lo, __shfl_xor_sync(0xffffffffu, h_lo, o));
    h_hi = max(h_hi, __shfl_xor_sync(0xffffffffu, h_hi, o));
  }
  const int t_first = h_lo / kKeys, t_end = (h_hi + kKeys - 1) / kKeys;  // (nothing seen: t_end is 0)
  int lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = __shfl_sync(0xffffffffu, r_lo, tq + 8 * i);
    hi[i] = __shfl_sync(0xffffffffu, r_hi, tq + 8 * i);
  }
  float slope2 = 0.f;
  if (p.mod.slopes) slope2 = dev::slope_at(p.mod, (int)(rb / p.B) * p.hp + j, p.n_head, p.status);

  for (int i = threadIdx.x; i < kRows * (D / 4); i += 32 * kWarps) {
    const int r = i / (D / 4), c = i % (D / 4);
    const long long off = q_base + (long long)(q0 + r) * p.hp * D + c * 4;
    const bool get = q0 + r < p.S && in_range(p.status, off, 4, p.qo_n);
    *reinterpret_cast<float4 *>(sQ + r * T::ldQ + c * 4) =
        get ? __ldg(reinterpret_cast<const float4 *>(p.q + off)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto fetch = [&](const float *src, float *dst, int ld, int t) {
    for (int i = lane; i < kKeys * (D / 4); i += 32) {
      const int r = i / (D / 4), c = i % (D / 4), key = t * kKeys + r;
      const long long off = kv_base + (long long)key * p.kvp * D + c * 4;
      const bool get = key < p.S && in_range(p.status, off, 4, p.kv_n);
      cp16(dst + r * ld + c * 4, src + (get ? off : 0), get);
    }
    cp_commit();
  };
  int t = t_first + warp;
  if (t < t_end) {
    fetch(p.k, sK, T::ldK, t);
    fetch(p.v, sV, D, t);
  }
  __syncthreads();

  float m[4], l[4];
  float2 acc[4][2 * nD];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * nD; ++e) acc[i][e] = make_float2(0.f, 0.f);
  }
  for (; t < t_end; t += kWarps) {
    const int k0 = t * kKeys;
    cp_wait<1>();  // K has landed (V is the later group)
    __syncwarp();
    float2 s2[4][nJ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int jj = 0; jj < nJ; ++jj) s2[i][jj] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 q4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q4[i] = *reinterpret_cast<const float4 *>(sQ + (tq + 8 * i) * T::ldQ + d);
#pragma unroll
      for (int jj = 0; jj < nJ; ++jj) {
        const float4 k4 = *reinterpret_cast<const float4 *>(sK + (tk + 4 * jj) * T::ldK + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s2[i][jj] = fma2(make_float2(q4[i].x, q4[i].y), make_float2(k4.x, k4.y), s2[i][jj]);
          s2[i][jj] = fma2(make_float2(q4[i].z, q4[i].w), make_float2(k4.z, k4.w), s2[i][jj]);
        }
      }
    }
    __syncwarp();  // K has been read
    if (t + kWarps < t_end)
      fetch(p.k, sK, T::ldK, t + kWarps);
    else
      cp_commit();  // (an empty group keeps the count)
    float s[4][nJ];
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int jj = 0; jj < nJ; ++jj) {
        s[i][jj] = s2[i][jj].x + s2[i][jj].y;
        big = fmaxf(big, fabsf(s[i][jj]));
      }
    if (p.mod.cap_out > 0.f) {
      if (__any_sync(0xffffffffu, big * big > p.mod.lim4)) {
        const dev::CapAny cap(p.mod);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int jj = 0; jj < nJ; jj += 4) {
            dev::f2x x = dev::f2_of(s[i][jj], s[i][jj + 1]), y = dev::f2_of(s[i][jj + 2], s[i][jj + 3]);
            uint32_t seen = 0;  // (what is unseen may be NaN, and four scores share a reciprocal)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const int key = k0 + tk + 4 * (jj + n);
              if (key >= lo[i] && key < hi[i]) seen |= 1u << n;
            }
            cap.drop_unseen(x, y, seen);
            cap(x, y);
            const float2 x2 = dev::f2_to(x), y2 = dev::f2_to(y);
            s[i][jj] = x2.x, s[i][jj + 1] = x2.y, s[i][jj + 2] = y2.x, s[i][jj + 3] = y2.y;
          }
      } else {
        const dev::Poly<4> long_form(p.mod.c4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int jj = 0; jj < nJ; jj += 2) {
            const dev::f2x x = dev::f2_of(s[i][jj], s[i][jj + 1]);
            const float2 y = dev::f2_to(dev::f2_mul(x, long_form(dev::f2_mul(x, x))));
            s[i][jj] = y.x, s[i][jj + 1] = y.y;
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < nJ; ++jj) s[i][jj] *= p.scale_log2;
    }
    if (p.mod.slopes) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < nJ; ++jj)
          s[i][jj] = fmaf(-slope2, fabsf((float)(k0 + tk + 4 * jj - (q0 + tq + 8 * i))), s[i][jj]);
    }
    float alpha[4];
    bool moved = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int jj = 0; jj < nJ; ++jj) {
        const int key = k0 + tk + 4 * jj;
        if (key < lo[i] || key >= hi[i]) s[i][jj] = -INFINITY;
        mx = fmaxf(mx, s[i][jj]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[i], mx);
      alpha[i] = m[i] == mn ? 1.f : ex2(m[i] - mn);  // (0 from -inf; both -inf: 1, of nothing)
      moved |= alpha[i] != 1.f;
      m[i] = mn;
      const float ref = mn == -INFINITY ? 0.f : mn;
      float sum = 0.f;
#pragma unroll
      for (int jj = 0; jj < nJ; ++jj) {
        const float e = ex2(s[i][jj] - ref);
        sum += e;
        sP[(tq + 8 * i) * T::ldP + tk + 4 * jj] = e;
      }
      l[i] = fmaf(l[i], alpha[i], sum);  // this lane's keys only; the four are added at the end
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 2 * nD; ++e) acc[i][e] = mul2(acc[i][e], make_float2(alpha[i], alpha[i]));
    }
    cp_wait<1>();  // V has landed (the next K is the later group)
    __syncwarp();  // ... for every lane, and P is written
#pragma unroll 4
    for (int k = 0; k < kKeys; k += 4) {
      float pr[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(sP + (tq + 8 * i) * T::ldP + k);
        pr[i][0] = v.x, pr[i][1] = v.y, pr[i][2] = v.z, pr[i][3] = v.w;
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int e = 0; e < nD; ++e) {
          const float4 v = *reinterpret_cast<const float4 *>(sV + (k + kk) * D + 16 * e + 4 * tk);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 pp = make_float2(pr[i][kk], pr[i][kk]);
            acc[i][2 * e] = fma2(pp, make_float2(v.x, v.y), acc[i][2 * e]);
            acc[i][2 * e + 1] = fma2(pp, make_float2(v.z, v.w), acc[i][2 * e + 1]);
          }
        }
    }
    __syncwarp();  // V and P have been read
    if (t + kWarps < t_end)
      fetch(p.v, sV, D, t + kWarps);
    else
      cp_commit();
  }
  cp_wait<0>();
  __syncwarp();
  // join the warps: their rows of O over K and V, the maxima and sums beside
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    const int r = tq + 8 * i;
#pragma unroll
    for (int e = 0; e < nD; ++e)
      *reinterpret_cast<float4 *>(mine + r * D + 16 * e + 4 * tk) =
          make_float4(acc[i][2 * e].x, acc[i][2 * e].y, acc[i][2 * e + 1].x, acc[i][2 * e + 1].y);
    if (tk == 0) sM[warp * kRows + r] = m[i], sL[warp * kRows + r] = l[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * (D / 4); i += 32 * kWarps) {
    const int r = i / (D / 4), c = i % (D / 4), row = q0 + r;
    if (row >= p.S) continue;
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sM[w * kRows + r]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mm != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = ex2(sM[w * kRows + r] - mm);
        const float4 v = *reinterpret_cast<const float4 *>(smem + T::kQ + w * T::kWarpFloats + r * D + c * 4);
        ll = fmaf(a, sL[w * kRows + r], ll);
        o.x = fmaf(a, v.x, o.x), o.y = fmaf(a, v.y, o.y), o.z = fmaf(a, v.z, o.z), o.w = fmaf(a, v.w, o.w);
      }
    }
    const float inv = ll > 0.f ? 1.f / ll : 0.f;  // a row that sees nothing: O = 0, LSE = -inf
    const long long off = q_base + (long long)row * p.hp * D + c * 4;
    if (in_range(p.status, off, 4, p.qo_n))
      *reinterpret_cast<float4 *>(p.o + off) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (c == 0 && in_range(p.status, hid * p.S + row, 1, p.lse_n))
      p.lse[hid * p.S + row] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994530942f : -INFINITY;
  }
}

template <int D>
cudaError_t launch_d(const SimtParams &sp, unsigned blocks, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(attn_fwd_mod_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)Tile<D>::kBytes);
  if (e != cudaSuccess) return e;
  attn_fwd_mod_simt_kernel<D><<<blocks, 32 * kWarps, Tile<D>::kBytes, st>>>(sp);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd_mod_simt(const ulysses_problem &p, const float *q, const float *k, const float *v,
                                     float *o, float *lse, uint32_t *status, const ulysses_score_mod &mod,
                                     cudaStream_t st) {
  SimtParams sp{};
  sp.q = q, sp.k = k, sp.v = v, sp.o = o, sp.lse = lse;
  sp.S = p.S, sp.B = p.B, sp.n_head = p.n_head;
  sp.hp = p.n_head / p.P, sp.kvp = kv_per_rank(p), sp.group = sp.hp / sp.kvp;
  sp.causal = p.causal;
  const float scale = p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf((float)p.head_dim);
  sp.scale_log2 = scale * 1.4426950408889634f;
  sp.status = status;
  sp.qo_n = (long long)p.B * p.S * p.n_head * p.head_dim;
  sp.kv_n = (long long)p.P * p.B * p.S * sp.kvp * p.head_dim;
  sp.lse_n = (long long)p.B * p.n_head * p.S;
  sp.mod = score_mod(p, mod);
  const long long blocks = (long long)((p.S + kRows - 1) / kRows) * p.P * p.B * sp.hp;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  switch (p.head_dim) {
    case 32: return launch_d<32>(sp, (unsigned)blocks, st);
    case 64: return launch_d<64>(sp, (unsigned)blocks, st);
    case 128: return launch_d<128>(sp, (unsigned)blocks, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ulysses
