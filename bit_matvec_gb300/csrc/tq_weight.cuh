// tq_weight.cuh -- exp((l - m) / T) as a 64-bit integer in units of 2^-45, good
// to 2^-36 of its value.
//
// A draw compares sums of up to 2^18 weights with a border. In 32 bits a sum is
// off by some 2^-24 of the total and a border is as near as the smallest
// weights, so one row in a hundred would draw a neighbour; the weights are
// therefore kept to 2^-36, and summed as integers, whose sums are exact in any
// order.
//
// With c = log2(e) / T, 2^((l - m) c) = 2^e T[j] 2^r for the exponent's integer
// part e, 11 bits j and the rest |r| <= 2^-12; T is a table of 2^(j / 2048) as
// the sum of two floats, and 2^r - 1 = y + y^2 / 2 for y = r ln 2, short by
// y^3 / 6 <= 2^-40. The difference and its product with c are kept as sums of
// two floats.
#pragma once

#include "tq_internal.cuh"

namespace tq {

constexpr int kWeightBits = 45;      // units of 2^-45
constexpr int kExpSteps = 2048;      // entries of the table

struct ExpTable {
  float2 v[kExpSteps];               // 2^(40 + j / kExpSteps) as a sum
};

// 2^x for 0 <= x < 1 in 64 bits, by the series of exp.
constexpr double exp2_series(double x) {
  const double y = x * 0.69314718055994530942;
  double sum = 1.0;
  for (int n = 24; n > 0; --n) sum = 1.0 + sum * y / n;
  return sum;
}
constexpr ExpTable make_exp_table() {
  ExpTable t = {};
  for (int j = 0; j < kExpSteps; ++j) {
    const double x = exp2_series((double)j / kExpSteps) * 1099511627776.0;
    t.v[j].x = (float)x;
    t.v[j].y = (float)(x - (double)t.v[j].x);
  }
  return t;
}

// What the weights of a row are relative to.
struct Weigher {
  float m, c_hi, c_lo;
  const float2* table;

  __device__ __forceinline__ uint64_t operator()(float l) const {
    const float d = l - m, b = d - l;
    const float dl = (l - (d - b)) - (m + b);       // d + dl = l - m exactly
    const float p = d * c_hi;
    if (!(p > -46.0f)) return 0;                    // less than half a unit
    const float pl = fmaf(dl, c_hi, fmaf(d, c_lo, fmaf(d, c_hi, -p)));
    constexpr float kMagic = 6144.0f;               // 1.5 * 2^12: steps of 2^-11
    const float nm = p + kMagic;
    const float r = (p - (nm - kMagic)) + pl;
    const int n = __float_as_int(nm) - __float_as_int(kMagic);
    const float2 t = table[n & (kExpSteps - 1)];
    const float y = r * 0.693147180559945f;
    const int rest = __float2int_rn(fmaf(t.x, fmaf(0.5f * y, y, y), t.y));
    const uint64_t mant = (__float_as_uint(t.x) & 0x7fffffu) | 0x800000u;
    // up to 2^41, in units of 2^-40 of 2^e; e <= 0
    const uint64_t w = (mant << 17) + (int64_t)rest;
    const int e = -(n >> 11);
    return e == 0 ? w << 5 : ((w << 5) + (uint64_t(1) << (e - 1))) >> e;
  }
};

// Floats as integers of the same order (both zeros alike).
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

}  // namespace tq
