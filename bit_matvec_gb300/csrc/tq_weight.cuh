// tq_weight.cuh -- exp(l / T) relative to a row's largest as a 64-bit integer, good to 2^-35 of its
// value and half a unit.
//
// A draw compares sums of up to 2^18 weights with a border. In 32 bits a sum is off by some 2^-24 of
// the total and a border is as near as the smallest weights, so one row in a hundred would draw a
// neighbour; the weights are therefore kept to 2^-35, and summed as integers, whose sums are exact in
// any order. 64-bit floats would do too, but run at 1/64 of the rate.
//
// With c = log2(e) / T, the weight is 2^(l c - R), R a multiple of 2^-11 just above the largest l c,
// plus one. l c is the sum of two floats (a product and its error), and its distance q from the
// nearest multiple of 2^-11 is exact in the first of them: adding K = 6144 - R rounds to such
// multiples, since 4096 <= l c + K < 8192, and leaves -e + j / 2048 in the sum's bits. The weight is
// then 2^-e T[j] 2^q with |q| <= 2^-12; T is a table of 2^(j / 2048) as the sum of two floats, and
// 2^q - 1 = q ln 2 + (q ln 2)^2 / 2, short by (q ln 2)^3 / 6 <= 2^-40.
//
// The unit is 2^-46 of 2^R, so a weight is at most 2^45 and 2^18 of them fit in 64 bits. Where bits
// fall off at the low end the last bit is set: off by at most one unit, to both sides alike, in one
// operation.
#pragma once

#include "tq_internal.cuh"

namespace tq {

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

struct Weigher {
  float c_hi, c_lo;    // log2(e) / T
  float k;             // 6144 - R
  float m;             // the largest logit
  float least;         // logits below weigh nothing
  int far;             // l c passes 2000: differences from m in its place
  const float2* table;

  static constexpr int kMagic = 0x45c00000;   // the bits of 6144.0f

  // For the row's largest logit (finite) and temperature.
  __device__ __forceinline__ void set(float top, float temp, const float2* t) {
    const double c = 1.4426950408889634074 / (double)temp;
    c_hi = (float)c;
    c_lo = (float)(c - (double)c_hi);
    m = top;
    table = t;
    const double e = (double)top * c;
    far = !(fabs(e) < 2000.0);
    const double r = far ? 1.0 : ceil(e * 2048.0) * (1.0 / 2048.0) + 1.0;
    k = (float)(6144.0 - r);
    least = fminf((float)(far ? (double)top - 46.0 / c : (r - 47.0) / c), top);
  }
  // The argument of the exponential as a float and what it lacks. (Operations by
  // name: a token has the same weight and bin wherever they are computed, which
  // a multiplication and addition that the compiler may join would not give.)
  __device__ __forceinline__ float exponent(float l, float& rest) const {
    if (!far) {
      const float p = __fmul_rn(l, c_hi);
      rest = __fmaf_rn(l, c_lo, __fmaf_rn(l, c_hi, -p));
      return p;
    }
    const float d = __fsub_rn(l, m), b = __fsub_rn(d, l);
    const float dl = __fsub_rn(__fsub_rn(l, __fsub_rn(d, b)), __fadd_rn(m, b));   // d + dl = l - m exactly
    const float p = __fmul_rn(d, c_hi);
    rest = __fmaf_rn(dl, c_hi, __fmaf_rn(d, c_lo, __fmaf_rn(d, c_hi, -p)));
    return p;
  }
  // l >= least. `top16`: the weight's leading 16 bits, its power of two apart.
  __device__ __forceinline__ uint64_t operator()(float l, uint32_t* top16 = nullptr) const {
    float rest;
    const float p = exponent(l, rest), nm = __fadd_rn(p, k);
    const float q = __fadd_rn(__fsub_rn(p, __fsub_rn(nm, k)), rest);
    const int bits = __float_as_int(nm);
    const float2 t = table[bits & (kExpSteps - 1)];
    constexpr float kLn2 = 0.693147180559945f, kHalfSquare = 0.240226506959101f;
    const int low = __float2int_rn(__fmaf_rn(__fmul_rn(t.x, q), __fmaf_rn(q, kHalfSquare, kLn2), t.y));
    const uint32_t mant = (__float_as_uint(t.x) & 0x7fffffu) | 0x800000u;
    const uint64_t w = ((uint64_t)mant << 17) + (int64_t)low;      // about 2^40 .. 2^41
    if (top16) *top16 = (uint32_t)(w >> 25);
    const int e = (kMagic >> 11) - (bits >> 11);                   // at least 1
    return ((w << 6) >> e) | (e > 6 ? 1u : 0u);
  }
  // The weight's place among 32 to an octave, falling; a rising logit never rises in it.
  __device__ __forceinline__ int bin(float l) const {
    float rest;
    const float nm = __fadd_rn(exponent(fmaxf(l, least), rest), k);
    return (kMagic >> 6) - (__float_as_int(nm) >> 6);
  }
};
constexpr int kWeightBins = 1536;    // 47 octaves and a little

// Floats as integers of the same order (both zeros alike), and back.
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

}  // namespace tq
