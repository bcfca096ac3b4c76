// The input-gradient product's operands.
//
// dx[m,k] = sum over rows n of z[m,n] T[n,k], z the gradient of row n's
// pre-activation times alpha[n], runs on the fp16 matrix cores: T is exact
// there and z is written as one fp16 term (relative rounding 2^-11, an
// eighth of the rounding a bf16 result gets anyway) or, for fp16 and fp32
// results, as two, high and low, which together keep 22 bits.  fp16 has the
// digits but not the range, so each token's z is scaled by a power of two
// (exact) that puts a bound on |z| at 2^15.  The bound is known before any z:
//   pre-activation <= P = s_x sum|q| max|alpha| + max(bias, 0),
//   |act'| <= 1.25 (2 P for relu2, where it is not 0), |act| <= P (P^2 for
//   relu2).  A bias that closes its output, however far below 0, so leaves
//   the others' scale alone.
// What the bound cannot know is which of its factors meet: the largest |z| of a
// token lies 2^4 .. 2^14 below it where scales and gradients are of one size
// (K up to 16384),
// and any number of powers of two where a row scale or a column of gradients
// far above the others belongs to an output whose gradient is 0.  A value is
// off by up to 2^-25 after scaling (half of fp16's least step), so S powers of
// two of slack make that 2^(S - 39) of the token's largest |z|.  The first pass
// therefore also finds each token's largest |z|, and where S is above
// kMostSlack, which leaves 2^-16 (one term) or 2^-24 (two), a second pass
// writes the token's z again under the scale that its largest asks for.
#pragma once

#include "sherry_launch.h"
#include "sherry_types.h"

namespace sherry {

// e such that |z| 2^e <= 2^15 for every z of a token: rows = (max |dy|,
// sum |q|), tops = (max |alpha|, max |alpha2|, max(bias, 0)), the maxima over
// finite values: an infinite or NaN gradient is one whatever the scale.
__device__ __forceinline__ int grad_exponent(float2 row, float s_x, const float* tops, int act, bool glu) {
  const double dy = row.x, sum = (double)row.y * fabs((double)s_x);
  const double a1 = tops[0], a2 = tops[1], pre = sum * a1 + (glu ? 0.0 : (double)tops[2]);
  const double slope = act == SHERRY_ACT_RELU2 ? 2.0 * pre : 1.25;
  const double bound = glu ? dy * slope * a1 * sum * a2 : dy * slope * a1;
  if (!(bound > 0.0)) return 0;
  if (bound > 1e300) return -120;
  const int e = 15 - (ilogb(bound) + 1);
  return e < -120 ? -120 : e > 120 ? 120 : e;
}

// The same, given the bits of the largest |z| (0: none known; infinite: the
// token's dx has no finite value): the exponent that z is left under.
constexpr int kMostSlack[2] = {23, 15};   // with one term, with two
__device__ __forceinline__ int exponent_used(int bound, uint32_t largest, int terms) {
  if (largest == 0u || largest >= 0x7F800000u) return bound;
  const int own = 14 - ilogbf(__builtin_bit_cast(float, largest));   // |z| 2^own < 2^15
  if (own - bound <= (terms == 2 ? kMostSlack[1] : kMostSlack[0])) return bound;
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
