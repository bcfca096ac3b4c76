// The input-gradient product's operands.
//
// dx[m,k] = sum over rows n of z[m,n] T[n,k], z the gradient of row n's
// pre-activation times alpha[n], runs on the fp16 matrix cores: T is exact
// there and z is written as one fp16 term (relative rounding 2^-11, an
// eighth of the rounding a bf16 result gets anyway) or, for fp16 and fp32
// results, as two, high and low, which together keep 22 bits.  fp16 has the
// digits but not the range, so each token's z is scaled by a power of two
// (exact) that puts its size at 2^15 at most.  That size is known before any z:
//   pre-activation <= P = s_x S max|alpha| + max(bias, 0),
//   |act'| <= 1.25 (2 P for relu2, where it is not 0), |act| <= P (P^2 for
//   relu2).  A bias that closes its output, however far below 0, so leaves
//   the others' scale alone.
// With S = sum|q| this is a bound, but one that lies sqrt(K) / 4 above what sums
// of K terms reach, twice over in the gated relu2.  S is therefore kSpread
// standard deviations of a sum with signs at random, sqrt(3/4 sum q^2), where
// that is less.  Nor can it know which of its factors meet: the largest |z| of a
// token lies 2 to 2^9 below it where scales and gradients are of one size, and
// any number of powers of two where a row scale or a column of gradients far
// above the others belongs to an output whose gradient is 0.  A value is off by
// up to 2^-25 after scaling (half of fp16's least step), so S powers of two of
// slack make that 2^(S - 39) of the token's largest |z|.  The first pass
// therefore also finds each token's largest |z|.  Where that passes 2^15, or
// where S is above kMostSlack, which leaves 2^-16 (one term) or 2^-24 (two), a
// second pass writes the token's z again under the scale that its largest
// asks for.
#pragma once

#include "sherry_launch.h"
#include "sherry_types.h"

namespace sherry {

constexpr float kSpread = 8.0f;

// e such that |z| 2^e <= 2^15 for every z of a token if S bounds its sums: tops =
// (max |alpha|, max |alpha2|, max(bias, 0)), the maxima over finite values: an
// infinite or NaN gradient is one whatever the scale.
__device__ __forceinline__ int grad_exponent(const GradRow& row, float S, float s_x, const float* tops, int act,
                                             bool glu) {
  const double dy = row.dy, sum = (double)S * fabs((double)s_x);
  const double a1 = tops[0], a2 = tops[1], pre = sum * a1 + (glu ? 0.0 : (double)tops[2]);
  const double slope = act == SHERRY_ACT_RELU2 ? 2.0 * pre : 1.25;
  const double bound = glu ? dy * slope * a1 * sum * a2 : dy * slope * a1;
  if (!(bound > 0.0)) return 0;
  if (bound > 1e300) return -120;
  const int e = 15 - (ilogb(bound) + 1);
  return e < -120 ? -120 : e > 120 ? 120 : e;
}

// That of the first pass.
__device__ __forceinline__ int first_exponent(const GradRow& row, float s_x, const float* tops, int act, bool glu) {
  return grad_exponent(row, row.likely, s_x, tops, act, glu);
}

// The exponent that z is left under, given the first pass's and the bits of the
// largest |z| it found.  An infinite one leaves the token's dx without a finite
// value; the bound then keeps the finite z from becoming infinite too.
constexpr int kMostSlack[2] = {23, 15};   // with one term, with two
__device__ __forceinline__ int last_exponent(int first, uint32_t largest, const GradRow& row, float s_x,
                                             const float* tops, int act, bool glu, int terms) {
  if (largest == 0u) return first;
  if (largest >= 0x7F800000u) return grad_exponent(row, row.sum, s_x, tops, act, glu);
  const int own = 14 - ilogbf(__builtin_bit_cast(float, largest));   // |z| 2^own < 2^15
  if (own >= first && own - first <= (terms == 2 ? kMostSlack[1] : kMostSlack[0])) return first;
  return own > 120 ? 120 : own;
}

__device__ __forceinline__ float exp2_of(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// v as one fp16 term, or as a high and a low one `stride` elements apart.
__device__ __forceinline__ void store_terms(_Float16* p, f4 v, int terms, int stride) {
  const h4 hi = __builtin_convertvector(v, h4);
  *reinterpret_cast<h4*>(p) = hi;
  if (terms == 2) {
    f4 rest = v - __builtin_convertvector(hi, f4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(fabsf(rest[i]) < 65536.0f)) rest[i] = 0.0f;   // an infinite or NaN high term stands alone
    *reinterpret_cast<h4*>(p + stride) = __builtin_convertvector(rest, h4);
  }
}

}  // namespace sherry
