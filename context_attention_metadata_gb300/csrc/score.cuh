// What happens to an attention score between the product and the softmax, beyond the scale: a
// soft cap and a bias by distance, shared by the forward and the backward kernel.
//
// With x = q . k from the tensor core, in base-2 units (times log2 e):
//   no cap   s = x * scale * log2 e
//   cap c    s = c * log2 e * tanh(x * scale / c)
//   bias     s -= slope_h * log2 e * |pos_q - pos_k|
// and for the gradient of a capped score ds/dx = scale * (1 - tanh^2), the factor 1 - tanh^2 here.
//
// With y = x scale / c, tanh y is taken in one of these ways, decided per warp and tile:
//   |y| <= 0.875 for all of the warp's scores: an odd polynomial, y (a0 + a1 y^2 + ... + a5 y^10),
//     the minimax fit of tanh(y) / y in y^2 over [0, 0.875^2] (computed by the exchange
//     algorithm), relative error 2^-22.7.  Its coefficients are folded with the scale on the
//     host, so that a capped score costs seven multiply-adds from x.
//   |y| <= 0.45, in the forward: the same with four terms, relative error 2^-22.
//   otherwise 1 - 2 / (1 + e^(2 y)): two calls to the special function unit, which also has the
//     softmax's exp2 to do, and an absolute error of 2^-22 c.  That is the rounding of a score
//     above 0.875 c, but the warp's other scores may be far smaller: where it would be more than
//     2^-14 (kWideCap), a score with |y| <= 0.875 takes the polynomial here too, score by score.
// The bias has no part in this choice: whether it is linear over the tile (the tile off the
// diagonal block, and no position track) decides only how the distances are had.
// The special function unit is what these two spare: an SM takes 32 exp2 or 16 reciprocals a
// clock (measured), 125 multiply-adds, and the softmax's exp2 takes one a score.  A forward over
// 64K packed tokens (16 heads of 128) takes 1667 us without a cap, 1597 with nearly every tile
// within the four-term range (cap 50), 1770 within the six-term one (cap 18), 2290 where most
// tiles go through the exponential (cap 5); the dK/dV kernel 3040, 3630, 3610 and 4300 us.  A
// polynomial in y instead of x needs one multiplication more a score: 3 to 9% slower.
// Folded coefficients leave fp32's range for caps far from the scores' size; set_cap then lowers
// the first two ways' limits to where the lost terms do not matter.
#pragma once

#include <math.h>

#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace marble {

// bits of a kernel's score variant; kScoreFixed (forward, with a cap alone): see kFixedCap
enum : int { kScoreCap = 1, kScoreBias = 2, kScoreFixed = 4 };

// A capped score without a bias lies in [-cap2, cap2], so the softmax needs no running maximum:
// where cap2 is at most kFixedCap, every row's stabiliser is 2^0.  A row's largest weight is then
// between 2^-80 and 2^80, and the middle of fp32's range is what is left to the values: sums over
// a row of values up to 2^47 / its keys stay finite in a row whose scores all are +cap, and values
// down to 2^-50 keep their bits in one whose scores all are -cap (a product of 2^-130 has 19 of
// fp32's, which the tensor core keeps below its normal range too).
// A bias with a slope >= 0 only lowers scores, and not that of a row's own key, which is legal in
// every row that has a legal key.  So the same holds for launches whose lists have the rows' own
// blocks (the fused ring, every needed block, the step of a shard with itself), decided for each
// head on the device; a step between different shards may hold nothing but far keys, all of whose
// weights 2^s can be below fp32's range, and keeps the running maximum.  (A piece of a row
// without the own key may lose its weights, which beside that key's are below 2^-46.)
// Saved are the maximum, its exchange between the two warps of a row and the rescaling (forward of
// 64K packed tokens, 16 heads of 128: cap 60, which keeps them, 1977 us, cap 50 1597; with a bias
// 2600 and 2045).
constexpr float kFixedCap = 80.f;

// cap2 above which a small score must not take the exponential's absolute error, 2^-22 cap2 (at
// 256 a weight is off by 2^-14 of itself, a 64th of its rounding to bf16)
constexpr float kWideCap = 256.f;

// tanh(y) / y in y^2: over |y| <= 0.875, and over |y| <= 0.45
__host__ __device__ constexpr double tanh_coef(int i) {
  constexpr double a[6] = {0.9999998509502919,   -0.33331914077818203, 0.1331109766192674,
                           -0.0526657826506247,  0.018277444003715584, -0.003840352757762384};
  return a[i];
}
constexpr double kTanhNear[4] = {0.9999997567401877, -0.3332946719023316, 0.13236369052147212,
                                 -0.0460281937984787};

struct ScoreParams {
  float c[6];             // s = x (c[0] + c[1] x^2 + ... + c[5] x^10) for |x| <= lim
  float lim;
  float cn[4];            // the same with four terms, |x| <= lim_n
  float lim_n;
  float ky;               // e^(2 y) = 2^(ky x)
  float cap2;             // cap * log2 e
  float neg_inv_cap2_sq;  // -1 / cap2^2
  float y_of_x;           // scale / cap
  int wide;               // cap2 > kWideCap
  const float* slopes;    // [hq] or null
  int bias_fixed;         // cap2 <= kFixedCap, and the launch's lists hold the rows' own blocks
  int consecutive;        // set for every variant: the positions of a block's tokens are consecutive
};

// the score variant a call needs
inline int score_bits(const marble_score_t* s) {
  return s ? (s->cap > 0.f ? kScoreCap : 0) | (s->slopes ? kScoreBias : 0) : 0;
}

// f(d, mod) with the head dim and the score variant as compile-time values
template <class F>
marble_status_t with_variant(int d, int mod, F f) {
  auto at_d = [&](auto dd) {
    switch (mod) {
      case 0: return f(dd, std::integral_constant<int, 0>{});
      case kScoreCap: return f(dd, std::integral_constant<int, kScoreCap>{});
      case kScoreBias: return f(dd, std::integral_constant<int, kScoreBias>{});
      default: return f(dd, std::integral_constant<int, kScoreCap | kScoreBias>{});
    }
  };
  if (d == 128) return at_d(std::integral_constant<int, 128>{});
  if (d == 64) return at_d(std::integral_constant<int, 64>{});
  return fail(MARBLE_ERR_UNSUPPORTED, "head dim must be 64 or 128");
}

// `cap` in [1e-30, 1e30]
inline void set_cap(ScoreParams* s, float cap, float scale) {
  double far[6];
  for (int i = 0; i < 6; ++i) far[i] = tanh_coef(i);
  const double log2e = 1.4426950408889634, k = (double)scale / cap, cap2 = cap * log2e;
  // c[i] = a[i] scale log2e k^(2i); returns the limit for |x|: `top` in y, less where a term is
  // lost below fp32's range (then up to where it is 2^-24 of the first), none where one is above
  // (and up to 1e18 for x and the score, whose squares are taken)
  auto fold = [&](const double* a, float* c, int terms, double top) {
    double f = scale * log2e;
    for (int i = 0; i < terms; ++i, f *= k * k) {
      c[i] = (float)(a[i] * f);
      if (!std::isfinite(c[i])) return -1.f;
      if (i > 0 && std::fabs(a[i] * f) < 1e-36)
        top = fmin(top, std::pow(0x1p-24 / std::fabs(a[i]), 0.5 / i));
    }
    return (float)fmin(top / k, 1e18 / fmax(1.0, scale * log2e));
  };
  s->lim = fold(far, s->c, 6, 0.875);
  s->lim_n = fold(kTanhNear, s->cn, 4, 0.45);
  s->ky = (float)(2.0 * log2e * k);
  s->cap2 = (float)cap2;
  s->y_of_x = (float)k;
  s->wide = s->cap2 > kWideCap;
  s->bias_fixed = s->cap2 <= kFixedCap;
  s->neg_inv_cap2_sq = (float)(-1.0 / (cap2 * cap2));
  if (!std::isfinite(s->neg_inv_cap2_sq)) s->lim = s->lim_n = -1.f;
}

// two fp32 values in a register pair and the packed operations on them: an instruction for two
// scores, where issuing instructions is what the elementwise warps run out of
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 x, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c[0] + c[1] x^2 + ... of a pair
template <int kTerms>
__device__ __forceinline__ F2 even_poly(F2 x, const float (&c)[kTerms]) {
  const F2 u = mul2(x, x);
  F2 r = f2(c[kTerms - 1]);
#pragma unroll
  for (int i = kTerms - 2; i >= 0; --i) r = fma2(r, u, f2(c[i]));
  return r;
}

// a pair's capped scores over its products: six terms, |x| <= lim, or four, |x| <= lim_n
template <int kTerms>
__device__ __forceinline__ F2 cap_factor(F2 x, const ScoreParams& p) {
  if constexpr (kTerms == 4)
    return even_poly(x, p.cn);
  else
    return even_poly(x, p.c);
}

// 1 / (1 + e^(2 y)): the capped score is cap2 (1 - 2 r), its slope's factor 4 r (1 - r)
__device__ __forceinline__ float cap_rcp(float x, const ScoreParams& p) {
  return fast_rcp(1.f + fast_exp2(x * p.ky));
}

// The capped scores of a pair by the exponential, and with kWide by it or the polynomial.
// rcp: the two 1 / (1 + e^(2 y)).  Whole warp.
template <bool kWide>
__device__ __forceinline__ F2 cap_far(float x0, float x1, const ScoreParams& p, float (&rcp)[2]) {
  rcp[0] = cap_rcp(x0, p);
  rcp[1] = cap_rcp(x1, p);
  float s0 = fmaf(-2.f * p.cap2, rcp[0], p.cap2), s1 = fmaf(-2.f * p.cap2, rcp[1], p.cap2);
  if constexpr (kWide) {
    // (in y, whose powers stay in range where the folded coefficients' do not)
    const F2 y = mul2(f2(x0, x1), f2(p.y_of_x));
    float y0, y1, t0, t1;
    split(y, &y0, &y1);
    if (__any_sync(0xffffffffu, fminf(fabsf(y0), fabsf(y1)) <= 0.875f)) {
      const F2 u = mul2(y, y);
      F2 t = f2((float)tanh_coef(5));
#pragma unroll
      for (int i = 4; i >= 0; --i) t = fma2(t, u, f2((float)tanh_coef(i)));
      split(mul2(mul2(t, y), f2(p.cap2)), &t0, &t1);
      s0 = fabsf(y0) <= 0.875f ? t0 : s0;
      s1 = fabsf(y1) <= 0.875f ? t1 : s1;
    }
  }
  return f2(s0, s1);
}

}  // namespace marble
