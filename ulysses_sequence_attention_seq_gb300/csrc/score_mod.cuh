// score_mod.cuh -- what the attention kernels do to a score between Q K^T and
// the softmax: cap it, bias it by distance, mask it.
//
//   s = scale q.k,  c = cap tanh(s / cap),  x = c - slope_h |i - k|,
//   key k seen by row i iff it lies in the row's interval (mask.cuh)
// The kernels work on base-2 logits x log2(e), so P = exp2(x - reference).
//
// tanh, y = s / cap.  The softmax warps are bound by the instructions they
// issue, so three forms, the first that all scores of a warp's tile allow:
//   |y| <= 1/4  y (a0 + a1 y^2 + a2 y^4), relative error 4.0e-7: three packed
//               instructions a pair of scores on top of the plain softmax's,
//   |y| <= 0.6  the same to y^8, 7.4e-8: five,
//   any         1 - 2 / (1 + exp(2 y)) with the hardware's exp2, and one
//               hardware reciprocal for four scores (of their product; so where
//               unseen keys of a forward give NaN, 0 is put for their scores).
// The polynomials interpolate tanh(sqrt z) / sqrt z at the Chebyshev points of
// the interval in z = y^2 and are applied to the raw q.k: scale, cap and
// log2(e) are in the coefficients.  The forward, which has its scores in
// registers throughout, keeps the form its row tile's earlier key tiles needed
// and looks at the sizes while it computes; a tile that needs a further form is
// done again in it (at most twice a row tile).  The backward looks first.  (The
// hardware's tanh is good to 2^-11 only: at a cap of 50 that moves a score by
// 0.02 and its probability by 2 %.)
#pragma once

#include <math.h>
#include <stdint.h>

#include "mask.cuh"
#include "sm100.cuh"

namespace ulysses {

// Template flags of these kernels: kModOn always, and what is done to a score.
// (With nothing on, the entry points call the plain attention's kernels.)
enum { kModOn = 1, kModCap = 2, kModBias = 4 };

namespace dev {

struct ScoreMod {
  MaskView mask;
  const float *slopes;  // [n_head] or null
  // scale / cap, cap * log2(e) and its inverse (cap_out 0: no cap)
  float cap_in, cap_out, inv_cap_out;
  // Raw scores whose squares are up to lim2 (lim4) may take the short (long)
  // polynomial: capped base-2 logit = s (c[0] + c[1] s^2 + ..); its slope
  // 1 - tanh^2 = f2[0] + f2[1] s^2 + .. (|y| <= 1/4, relative error 2.8e-6)
  float lim2, lim4;
  // (Aligned: they are constant operands, read in pairs.  Moved by a member before
  // them the capped forward took 1731 us instead of 1640.)
  alignas(16) float c2[3];
  alignas(16) float c4[5];
  alignas(16) float f2[3];
};

// Two floats in one 64-bit register pair, the operand of the packed float
// instructions.  (As such a pair, and not as two floats, a constant operand is
// put together once and stays so.)
typedef unsigned long long f2x;
__device__ __forceinline__ f2x f2_of(float a, float b) {
  f2x r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_to(f2x a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ f2x f2_fma(f2x a, f2x b, f2x c) {
  f2x d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2x f2_mul(f2x a, f2x b) {
  f2x d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2x f2_add(f2x a, f2x b) {
  f2x d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Both halves `a`, kept in registers from here on.
__device__ __forceinline__ f2x f2_const(float a) {
  f2x r = f2_of(a, a);
  asm("" : "+l"(r));
  return r;
}
// As sm100::tmem_ld32, 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

struct Nil {};
__device__ __forceinline__ float operator+(float a, Nil) { return a; }

// Coefficients c[0 .. N] of a polynomial in registers.
template <int N>
struct Poly {
  f2x c[N + 1];
  template <typename Zero>
  __device__ __forceinline__ Poly(const float (&from)[N + 1], Zero zero) {
#pragma unroll
    for (int i = 0; i <= N; ++i) c[i] = f2_const(from[i] + zero);
  }
  __device__ __forceinline__ explicit Poly(const float (&from)[N + 1]) : Poly(from, Nil()) {}
  __device__ __forceinline__ f2x operator()(f2x u) const {
    f2x a = c[N];
#pragma unroll
    for (int i = N - 1; i >= 0; --i) a = f2_fma(a, u, c[i]);
    return a;
  }
};

// 1 + exp(2 y) of two raw scores (k = 2 log2(e) cap_in), y cut at 10 (tanh is 1
// there; four such factors still multiply to a float).
__device__ __forceinline__ f2x one_plus_exp(f2x s, f2x k, f2x one) {
  float2 e = f2_to(f2_mul(s, k));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(e.x) : "f"(28.853900817779268f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(e.y) : "f"(28.853900817779268f));
  return f2_add(f2_of(sm100::ex2(e.x), sm100::ex2(e.y)), one);
}
// The exponential form: capped base-2 logits of four raw scores.
struct CapAny {
  f2x k, one, n, c;
  __device__ __forceinline__ explicit CapAny(const ScoreMod &m) : CapAny(m, Nil()) {}
  template <typename Zero>
  __device__ __forceinline__ CapAny(const ScoreMod &m, Zero zero)
      : k(f2_const(m.cap_in * 2.885390081777927f + zero)), one(f2_const(1.0f + zero)),
        n(f2_const(-2.0f * m.cap_out + zero)), c(f2_const(m.cap_out + zero)) {}
  __device__ __forceinline__ void operator()(f2x &s0, f2x &s1) const {
    const f2x a = one_plus_exp(s0, k, one), b = one_plus_exp(s1, k, one);
    const float2 t = f2_to(f2_mul(a, b));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t.x * t.y));
    const f2x r2 = f2_mul(f2_of(r, r), f2_of(t.y, t.x));  // 1 / (a.x b.x), 1 / (a.y b.y)
    s0 = f2_fma(f2_mul(r2, b), n, c);
    s1 = f2_fma(f2_mul(r2, a), n, c);
  }
  // 0 for those of four scores whose bit of `seen` is off: the others would take
  // NaN from the product that the reciprocal is of.
  static __device__ __forceinline__ void drop_unseen(f2x &s0, f2x &s1, uint32_t seen) {
    float2 a = f2_to(s0), b = f2_to(s1);
    if (!(seen & 1u)) a.x = 0.f;
    if (!(seen & 2u)) a.y = 0.f;
    if (!(seen & 4u)) b.x = 0.f;
    if (!(seen & 8u)) b.y = 0.f;
    s0 = f2_of(a.x, a.y), s1 = f2_of(b.x, b.y);
  }
};

// What form kForm of tanh (-1: none) needs in registers.  `zero` is Nil, or a 0
// from memory: where that is read inside a loop, there the registers are taken,
// not before it, for its whole length, by the coefficients of every form.  (dQ of
// 8K tokens x 32 heads of 64, capped: 675 -> 661 us.)
template <int kForm>
struct CapForm {
  const Poly<kForm == 1 ? 4 : 2> poly;
  template <typename Zero>
  __device__ __forceinline__ CapForm(const ScoreMod &m, Zero zero) : poly(pick(m), zero) {}
  static __device__ __forceinline__ auto pick(const ScoreMod &m) -> const float (&)[kForm == 1 ? 5 : 3] {
    if constexpr (kForm == 1)
      return m.c4;
    else
      return m.c2;
  }
};
template <>
struct CapForm<2> {
  const CapAny any;
  template <typename Zero>
  __device__ __forceinline__ CapForm(const ScoreMod &m, Zero zero) : any(m, zero) {}
};
template <>
struct CapForm<-1> {
  template <typename Zero>
  __device__ __forceinline__ CapForm(const ScoreMod &, Zero) {}
};
// The same with the slope f = 1 - tanh^2: a polynomial beside form 0's, else
// 1 - (c / cap)^2 of the capped logit c.
template <int kForm>
struct CapFormSlope : CapForm<kForm> {
  const f2x inv, ninv, one;
  template <typename Zero>
  __device__ __forceinline__ CapFormSlope(const ScoreMod &m, Zero zero)
      : CapForm<kForm>(m, zero), inv(f2_const(m.inv_cap_out + zero)), ninv(f2_const(-m.inv_cap_out + zero)),
        one(f2_const(1.f + zero)) {}
};
template <>
struct CapFormSlope<0> : CapForm<0> {
  const Poly<2> slope;
  template <typename Zero>
  __device__ __forceinline__ CapFormSlope(const ScoreMod &m, Zero zero) : CapForm<0>(m, zero), slope(m.f2, zero) {}
};
template <>
struct CapFormSlope<-1> : CapForm<-1> {
  using CapForm<-1>::CapForm;
};

// The largest square of the scores a thread holds.
template <int kRows>
__device__ __forceinline__ float largest_square(const uint32_t (&s)[kRows][32]) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const f2x v = f2_of(__uint_as_float(s[r][e]), __uint_as_float(s[r][e + 1]));
      const float2 u = f2_to(f2_mul(v, v));
      m[(e / 2) & 3] = sm100::max3(m[(e / 2) & 3], u.x, u.y);
    }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// The form that the largest squares of the raw scores of a warp's threads need.
__device__ __forceinline__ int cap_form(float big, const ScoreMod &m) {
  if (!__any_sync(0xffffffffu, big > m.lim2)) return 0;
  return __any_sync(0xffffffffu, big > m.lim4) ? 2 : 1;
}

// Raw scores on their way to the exponential form, where four share a
// reciprocal: if any of the warp's is NaN, 0 for those whose bit of `seen` is off
// (keys of padding may hold anything).
template <int n>
__device__ __forceinline__ void drop_unseen_nan(uint32_t (&s)[n], uint32_t seen) {
  f2x sum = f2_of(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < n; e += 2) sum = f2_add(sum, f2_of(__uint_as_float(s[e]), __uint_as_float(s[e + 1])));
  const float2 sum2 = f2_to(sum);
  const float all = sum2.x + sum2.y;  // (NaN of infinities of both signs, too)
  if (__any_sync(0xffffffffu, all != all)) {
#pragma unroll
    for (int e = 0; e < n; ++e)
      if (!(seen & (1u << e))) s[e] = 0u;
  }
}

// Head h's slope, for base-2 logits.
__device__ __forceinline__ float slope_at(const ScoreMod &m, int h, int n_head, uint32_t *status) {
  return in_range(status, h, 1, n_head) ? __ldg(m.slopes + h) * 1.4426950408889634f : 0.f;
}

// The bias -slope |lead + c| (base 2) of score c = 0, 1, ..: `lead` is the
// position of the first score a thread holds minus the fixed position of its
// row (or key), so key and query side read the same.  Linear in c, slope2 c +
// base, unless the diagonal crosses the warp's scores; `side` -1 (1) says that
// all scores that matter have lead + c <= 0 (>= 0).
struct LinearBias {
  bool ok;
  float slope2, base;
};
template <int n>
__device__ __forceinline__ LinearBias linear_bias(float slope2, int lead, int side = 0) {
  const bool below = side < 0 || __all_sync(0xffffffffu, lead + n - 1 <= 0);
  const bool above = side > 0 || __all_sync(0xffffffffu, lead >= 0);
  const float sl = below ? slope2 : -slope2;
  return {below || above, sl, sl * (float)lead};
}
// Its eight pairs c = 0 .. 15 without the base; pair e of the next sixteen
// scores is the same on a base 16 slope2 further.
struct BiasSteps {
  f2x d[8];
  __device__ __forceinline__ explicit BiasSteps(const LinearBias &b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = f2_of((float)(2 * e) * b.slope2, (float)(2 * e + 1) * b.slope2);
  }
};

// Bits [lo, hi) of a word (either may lie outside it).
__device__ __forceinline__ uint32_t bits_of(int lo, int hi) {
  const uint32_t below = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u;
  return lo <= 0 ? below : lo >= 32 ? 0u : below & (0xffffffffu << lo);
}

// Base-2 logits in place of the raw scores a thread holds, 32 to a row of `s`,
// any size, any side of the diagonal.  `part`: some of the warp's keys, outside
// [lo, hi), are not seen; what becomes of their scores does not matter, but it
// stays with them.
template <int kMod, int kRows>
__device__ __forceinline__ void logits(uint32_t (&s)[kRows][32], const ScoreMod &m, float scale_log2, float slope2,
                                       int lead, bool part, int lo, int hi) {
  const float lf = (float)lead;
  if constexpr ((kMod & kModCap) != 0) {
    // (The exponential form is off by some 2^-22 of the cap however small the
    // score is: a large cap needs the polynomial, which is not.)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float big = 0.f;
#pragma unroll
      for (int e = 0; e < 32; e += 2)
        big = sm100::max3(big, fabsf(__uint_as_float(s[r][e])), fabsf(__uint_as_float(s[r][e + 1])));
      if (__any_sync(0xffffffffu, big * big > m.lim4)) {
        const CapAny cap(m);
        if (part) drop_unseen_nan(s[r], bits_of(lo - 32 * r, hi - 32 * r));
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          f2x x = f2_of(__uint_as_float(s[r][e]), __uint_as_float(s[r][e + 1]));
          f2x y = f2_of(__uint_as_float(s[r][e + 2]), __uint_as_float(s[r][e + 3]));
          cap(x, y);
          const float2 x2 = f2_to(x), y2 = f2_to(y);
          s[r][e] = __float_as_uint(x2.x), s[r][e + 1] = __float_as_uint(x2.y);
          s[r][e + 2] = __float_as_uint(y2.x), s[r][e + 3] = __float_as_uint(y2.y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float x = __uint_as_float(s[r][e]), u = x * x;
          float a = fmaf(m.c4[4], u, m.c4[3]);
          a = fmaf(a, u, m.c4[2]);
          a = fmaf(a, u, m.c4[1]);
          s[r][e] = __float_as_uint(x * fmaf(a, u, m.c4[0]));
        }
      }
    }
  }
  if constexpr ((kMod & kModBias) != 0) {
    const float mul = (kMod & kModCap) ? 1.0f : scale_log2;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int e = 0; e < 32; ++e)
        s[r][e] =
            __float_as_uint(fmaf(__uint_as_float(s[r][e]), mul, -slope2 * fabsf(lf + (float)(32 * r + e))));
  }
}

}  // namespace dev

// Host: the kernel flags and parameters of a checked ulysses_score_mod.
inline int score_mod_flags(const ulysses_score_mod &m) {
  return kModOn | (m.softcap > 0.f ? kModCap : 0) | (m.slopes ? kModBias : 0);
}
inline dev::ScoreMod score_mod(const ulysses_problem &p, const ulysses_score_mod &m) {
  dev::ScoreMod s{};
  s.mask = mask_view(p, m.mask);
  s.slopes = m.slopes;
  if (m.softcap > 0.f) {
    const double scale = p.softmax_scale > 0.f ? p.softmax_scale : 1.0 / sqrt((double)p.head_dim);
    const double y = scale / m.softcap, out = m.softcap * 1.4426950408889634;
    s.cap_in = (float)y;
    s.cap_out = (float)out;
    s.inv_cap_out = (float)(1.0 / out);
    static const double t2[3] = {0.999999603463, -0.33321896989, 0.128414339271};
    static const double t4[5] = {0.999999925963, -0.333323020404, 0.133100644256, -0.0520966534081, 0.0154687513018};
    static const double g2[3] = {0.999997253807, -0.999207662195, 0.632507683902};
    // Scaled coefficients have to be normal floats.  Where the long form's are
    // not (large caps) the short form does for both, and where its are not either
    // the linear term alone, as far as |y| <= 1e-3: error y^2 / 3 = 3.3e-7.
    auto normal = [](double v) { return fabs(v) > 1e-36 && fabs(v) < 1e36; };
    double k = y;
    bool ok2 = true, ok4 = true;
    for (int i = 0; i < 5; ++i, k *= y * y) {
      ok4 = ok4 && normal(out * k * t4[i]);
      if (i < 3) ok2 = ok2 && normal(out * k * t2[i]) && normal(k / y * g2[i]);
    }
    k = y;
    for (int i = 0; i < 5; ++i, k *= y * y) {
      if (i < 3) s.c2[i] = ok2 || i == 0 ? (float)(out * k * (ok2 ? t2[i] : 1.0)) : 0.f;
      if (i < 3) s.f2[i] = ok2 || i == 0 ? (float)(k / y * (ok2 ? g2[i] : 1.0)) : 0.f;
      s.c4[i] = ok4 ? (float)(out * k * t4[i]) : i < 3 ? s.c2[i] : 0.f;
    }
    s.lim2 = (float)fmin((ok2 ? 0.062499 : 1e-6) / (y * y), 1e36);
    s.lim4 = ok4 ? (float)fmin(0.359999 / (y * y), 1e36) : s.lim2;
  }
  return s;
}

}  // namespace ulysses
