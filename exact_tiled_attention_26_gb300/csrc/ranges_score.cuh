// The cap of the scores, shared by the attention over ranges (forward, gradients) and the attention of drafted tokens.
#pragma once

#include "ptx.cuh"

namespace fa {

// cap tanh(s / cap) in base 2 for scores x before scaling (x = s / unit), made on the host.
//   tanh(s / cap) = 1 - 2 / (1 + 2^y), y = 2 log2 e s / cap
// in absolute error some 2^-22 whatever y is (2^y = infinity: 1; a NaN stays one).  Two operations of the
// special-function unit an element, three with the weight's exponential: at 16 a clock and SM they take 3 x 1024 clocks
// for a tile's 16384 scores, and bound a capped forward (16384 tokens, 32 + 8 heads, d = 128: 2.81 ms; uncapped 1.51).
// So that takes one reciprocal for four scores (cap_scores_fast, 2.40 ms).  The gradients and a decoded token are bound
// by other things and were slower with it (8192 tokens: 1.51 ms against 1.48).  Measured besides for the forward: one
// reciprocal for two 2.64; a polynomial of degree 13 where no score passes the cap 2.69, for every other pair 2.48.
struct CapArgs {
  float cap_log2;  // cap log2 e; 0: no cap
  float to_y;      // y = x to_y
};
// unit: what x is multiplied by to be a score s.
inline CapArgs cap_args(double cap, double unit) {
  constexpr double log2e = 1.4426950408889634;
  if (!(cap > 0.0)) return CapArgs{0.f, 0.f};
  return CapArgs{static_cast<float>(cap * log2e), static_cast<float>(2.0 * log2e * unit / cap)};
}

// x becomes the capped score in base 2.
template <int N>
FA_DEV void cap_scores(float (&x)[N], const CapArgs& c) {
  const uint64_t to2 = f2pack(c.to_y, c.to_y), cap2 = f2pack(c.cap_log2, c.cap_log2);
  const uint64_t m2 = f2pack(-2.f * c.cap_log2, -2.f * c.cap_log2), one2 = f2pack(1.f, 1.f);
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float y0, y1, a0, a1;
    f2unpack(fmul2(f2pack(x[k], x[k + 1]), to2), y0, y1);
    f2unpack(fadd2(f2pack(ex2(y0), ex2(y1)), one2), a0, a1);
    f2unpack(ffma2(f2pack(rcp(a0), rcp(a1)), m2, cap2), x[k], x[k + 1]);
  }
}

// The same for the gradients, with the cap's derivative:
//   tanh = +-(1 - 2 w), 1 - tanh^2 = 4 (w - w^2), w = 1 / (1 + 2^|y|),
// which keeps its relative precision however far a score is beyond the cap, as w <= 1/2 (of 1 - tanh^2 itself some 2^-23
// would be left there).  `rate` is the derivative times 1 / kRateScale: w^2 - w is one operation from -w.
constexpr float kRateScale = -4.f;
template <int N>
FA_DEV void cap_scores_rate(float (&x)[N], float (&rate)[N], const CapArgs& c) {
  const uint64_t to2 = f2pack(c.to_y, c.to_y), cap2 = f2pack(c.cap_log2, c.cap_log2);
  const uint64_t m2 = f2pack(2.f * c.cap_log2, 2.f * c.cap_log2), minus2 = f2pack(-1.f, -1.f);
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float y0, y1, a0, a1, s0, s1;
    f2unpack(fmul2(f2pack(x[k], x[k + 1]), to2), y0, y1);
    f2unpack(ffma2(f2pack(ex2(fabsf(y0)), ex2(fabsf(y1))), minus2, minus2), a0, a1);
    const uint64_t w = f2pack(rcp(a0), rcp(a1));  // -w
    f2unpack(ffma2(w, m2, cap2), s0, s1);
    x[k] = copysignf(s0, y0), x[k + 1] = copysignf(s1, y1);
    f2unpack(ffma2(w, w, w), rate[k], rate[k + 1]);
  }
}

// The same with one reciprocal for four scores: false if the products of four 1 + 2^y do not stay finite (scores of some
// ten times the cap, or a NaN, which would reach the others), then x is to be taken again with cap_scores.
template <int N>
FA_DEV bool cap_scores_fast(float (&x)[N], const CapArgs& c) {
  const uint64_t to2 = f2pack(c.to_y, c.to_y), one2 = f2pack(1.f, 1.f);
  float worst = 0.f;
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    float y[4], a[4];
    f2unpack(fmul2(f2pack(x[k], x[k + 1]), to2), y[0], y[1]);
    f2unpack(fmul2(f2pack(x[k + 2], x[k + 3]), to2), y[2], y[3]);
    f2unpack(fadd2(f2pack(ex2(y[0]), ex2(y[1])), one2), a[0], a[1]);
    f2unpack(fadd2(f2pack(ex2(y[2]), ex2(y[3])), one2), a[2], a[3]);
    const float p = a[0] * a[1], q = a[2] * a[3], all = p * q;
    worst = max_nan(worst, all);
    const float f = rcp(all) * (-2.f * c.cap_log2), fp = f * q, fq = f * p;
    x[k] = fmaf(fp, a[1], c.cap_log2), x[k + 1] = fmaf(fp, a[0], c.cap_log2);
    x[k + 2] = fmaf(fq, a[3], c.cap_log2), x[k + 3] = fmaf(fq, a[2], c.cap_log2);
  }
  return worst < 1e30f;
}

}  // namespace fa
