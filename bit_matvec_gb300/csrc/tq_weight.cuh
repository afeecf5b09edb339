// tq_weight.cuh -- exp(l / T) relative to a row's largest as a 64-bit integer, good to 2^-35 of its
// value and a unit.
//
// A draw compares sums of up to 2^18 weights with a border. In 32 bits a sum is off by some 2^-24 of
// the total and a border is as near as the smallest weights, so one row in a hundred would draw a
// neighbour; the weights are therefore kept to 2^-35, and summed as integers, whose sums are exact in
// any order. 64-bit floats would do too, but run at 1/64 of the rate.
//
// With c = log2(e) / T, the weight is 2^(l c - R), R a multiple of 2^-11 just above the largest l c,
// plus one. (Where that passes 2000, l is replaced by its difference from the largest, which is exact
// for every logit that weighs anything: the two are within a factor of two.) l c is the sum of two floats (a product and its error), and its distance q from the
// nearest multiple of 2^-11 is exact in the first of them: adding K = 6144 - R rounds to such
// multiples, since 4096 <= l c + K < 8192, and leaves -e + j / 2048 in the sum's bits. The weight is
// then 2^-e T[j] 2^q with |q| <= 2^-12; T is a table of 2^(j / 2048) as the sum of two floats, and
// 2^q - 1 = q ln 2 + (q ln 2)^2 / 2, short by (q ln 2)^3 / 6 <= 2^-40.
//
// The unit is 2^-54 of 2^R, so a weight is at most 2^53 and 2^10 of them fit in 64 bits: those of a list, of
// a block of 512, of a thread. Sums of more are in units of 2^-46, which 2^18 fit in. (With that unit for the
// weights as well, a quarter million of them a few units each were off by 2^-25 of the total together.)
// A weight is cut to its unit, so those of 2^-14 of 2^R and more lose nothing; those of 2^-6 and more are
// whole coarse units: where a share of equal logits is a whole number of them, it is met exactly.
#pragma once

#include "tq_tcgen05.cuh"

namespace tq {

constexpr int kExpSteps = 2048;      // entries of the table

struct alignas(16) ExpTable {
  float hi[kExpSteps], lo[kExpSteps];   // 2^(40 + j / kExpSteps) as a sum
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
    t.hi[j] = (float)x;
    t.lo[j] = (float)(x - (double)t.hi[j]);
  }
  return t;
}

constexpr int kWeightBins = 896;     // 16 to an octave, 54 octaves and more
constexpr int kOctaves = 54;         // a weight below 2^R by more is less than a unit
constexpr int kCoarse = 8;           // a coarse unit is 2^8 units

struct Weigher {
  float c_hi, c_lo;    // log2(e) / T
  float k;             // 6144 - R
  float shift;         // taken from every logit: 0, or the largest one
  float least;         // logits below weigh nothing
  const ExpTable* table;

  static constexpr int kMagic = 0x45c00000;   // the bits of 6144.0f
  static constexpr int kBinShift = 7;         // 2048 / 16 steps a bin

  // log2(e) / T as a sum, for a temperature of 2^-100 .. 2^100. (By 32-bit
  // operations, here and below: a block's 512 threads wait ten microseconds for
  // the same few in 64 bits.)
  __device__ __forceinline__ void set_temperature(float t) {
    constexpr float kHi = 1.44269504088896341f, kLo = (float)(1.44269504088896341 - (double)kHi);
    c_hi = __fdiv_rn(kHi, t);
    c_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-c_hi, t, kHi), kLo), t);
  }
  // For the row's largest logit (finite).
  __device__ __forceinline__ void set_top(float top, float t, const ExpTable* from) {
    table = from;
    const float p = __fmul_rn(top, c_hi), octave = __fmul_rn(t, 0.693147180559945f);
    const bool far = !(fabsf(p) < 2000.0f);
    shift = far ? top : 0.0f;
    // (one step more for what c_lo adds)
    const float r = far ? 1.0f : ceilf(p * 2048.0f) * (1.0f / 2048.0f) + (1.0f + 1.0f / 2048.0f);
    k = 6144.0f - r;
    least = fminf(far ? top - (kOctaves - 1) * octave : (r - kOctaves) * octave, top);
  }
  // The same with whole octaves: sums relative to other logits' are shifts
  // apart. Returns R; not for logits whose exponent passes 2000.
  __device__ __forceinline__ int set_octave(float top, const ExpTable* from) {
    table = from;
    shift = 0.0f;
    const float r = ceilf(__fmul_rn(top, c_hi)) + 2.0f;
    k = 6144.0f - r;
    least = -INFINITY;
    return (int)r;
  }
  // ln(w / total) for the weight of l and a sum in coarse units, 2^-46 of 2^(6144 - k).
  __device__ __forceinline__ float log_share(float l, uint64_t total) const {
    const float x = __fsub_rn(l, shift), p = __fmul_rn(x, c_hi);
    const float rest = __fmaf_rn(x, c_lo, __fmaf_rn(x, c_hi, -p));       // x c - p
    float whole, part;
    log2_of(total, *table, whole, part);
    // x c - R + 46 - log2(total): p and a multiple of 2^-11, and what they lack
    const float b = (6144.0f - k) - 46.0f + whole;
    const float a = __fsub_rn(p, b), t = __fsub_rn(a, p);
    const float lack = __fadd_rn(__fsub_rn(p, __fsub_rn(a, t)), -__fadd_rn(b, t));
    const float low = __fadd_rn(__fadd_rn(lack, rest), -part);
    constexpr float kLn2 = 0.69314718055994531f, kLn2Low = (float)(0.69314718055994531 - (double)kLn2);
    const float h = __fmul_rn(a, kLn2);
    return __fadd_rn(h, __fadd_rn(__fmaf_rn(a, kLn2, -h), __fmaf_rn(a, kLn2Low, __fmul_rn(low, kLn2))));
  }
  // log2 of a positive integer, as a multiple of 2^-11 and the rest,
  // good to 2^-34: the leading bits m over the table's entry below are 1 + d, d < 2^-10.
  static __device__ __forceinline__ void log2_of(uint64_t n, const ExpTable& t, float& whole, float& part) {
    const int zeros = __clzll((long long)n);
    const uint64_t m = n << zeros;
    const float hi = (float)(uint32_t)(m >> 40) * 0x1p17f;                     // 2^40 .. 2^41
    const float lo = (float)(uint32_t)((m >> 16) & 0xffffffu) * 0x1p-7f;
    const int j = max(0, min(kExpSteps - 1, (int)(__log2f(hi * 0x1p-40f) * kExpSteps)));
    const float d = __fdiv_rn(__fadd_rn(__fsub_rn(hi, t.hi[j]), __fsub_rn(lo, t.lo[j])), t.hi[j]);
    part = __fmul_rn(1.44269504088896341f, __fmaf_rn(__fmul_rn(d, d), __fmaf_rn(d, 1.0f / 3.0f, -0.5f), d));
    whole = (float)(63 - zeros) + (float)j * (1.0f / kExpSteps);
  }
  // N (even) weights, for logits of at least `least` (others give anything), and their bits: the
  // exponent in steps of 2^-11. Two at a time, an operation for both.
  template <int N> __device__ __forceinline__ void operator()(const float (&l)[N], uint64_t (&w)[N], int (&bits)[N],
                                                              uint32_t* lead = nullptr) const {
    using namespace tc;
    const uint64_t ch = f2_packf(c_hi, c_hi), minus_ch = f2_packf(-c_hi, -c_hi), minus_cl = f2_packf(-c_lo, -c_lo);
    const uint64_t kk = f2_packf(k, k), sh = f2_packf(shift, shift);
    constexpr float kLn2 = 0.693147180559945f, kHalfSquare = 0.240226506959101f;
    const uint64_t ln2 = f2_packf(kLn2, kLn2), half_square = f2_packf(kHalfSquare, kHalfSquare);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t x = f2_sub(f2_packf(l[i], l[i + 1]), sh);
      const uint64_t p = f2_mul(x, ch);
      const uint64_t over = f2_fma(x, minus_cl, f2_fma(x, minus_ch, p));    // p - x c
      const uint64_t nm = f2_add(p, kk);
      const uint64_t q = f2_sub(f2_sub(p, f2_sub(nm, kk)), over);
      bits[i] = (int)(uint32_t)nm;
      bits[i + 1] = (int)(uint32_t)(nm >> 32);
      const int j0 = bits[i] & (kExpSteps - 1), j1 = bits[i + 1] & (kExpSteps - 1);
      const float t0 = table->hi[j0], t1 = table->hi[j1];
      const float2 low = f2_unpack(f2_fma(f2_mul(f2_packf(t0, t1), q), f2_fma(q, half_square, ln2),
                                          f2_packf(table->lo[j0], table->lo[j1])));
      finish(t0, low.x, bits[i], w[i], lead ? lead + i : nullptr);
      finish(t1, low.y, bits[i + 1], w[i + 1], lead ? lead + i + 1 : nullptr);
    }
  }
  // T[j] as a 24-bit integer with what is to be added: about 2^40 .. 2^41, then 2^14 times that, cut to
  // its place.
  static __device__ __forceinline__ void finish(float t, float low, int bits, uint64_t& w, uint32_t* lead) {
    const uint32_t mant = (__float_as_uint(t) & 0x7fffffu) | 0x800000u;
    const uint64_t v = ((uint64_t)mant << 31) + (int64_t)__float2int_rn(low) * 16384;
    if (lead) *lead = (uint32_t)(v >> 42);
    w = v >> ((kMagic >> 11) - (bits >> 11));
  }
  __device__ __forceinline__ uint64_t one(float l) const {
    const float two[2] = {l, l};
    uint64_t w[2];
    int bits[2];
    (*this)(two, w, bits);
    return w[0];
  }
  // The weight's place among 16 to an octave, falling; a rising logit never rises in it. The same
  // operations as above: a token has the same bin wherever it is computed.
  __device__ __forceinline__ int bin(float l) const {
    return bin_of(__float_as_int(__fadd_rn(__fmul_rn(__fsub_rn(fmaxf(l, least), shift), c_hi), k)));
  }
  static __device__ __forceinline__ int bin_of(int bits) { return (kMagic >> kBinShift) - (bits >> kBinShift); }
  static __device__ __forceinline__ int octave_of(int bin) { return (bin + 15) / 16; }
};

// t ln(x) as a sum of two floats, for x > 0 (infinity gives infinity).
__device__ __forceinline__ void scaled_log(float x, float t, const ExpTable& table, float& hi, float& lo) {
  const uint32_t b = __float_as_uint(x);
  if (b >= 0x7f800000u) {
    hi = INFINITY;
    lo = 0.0f;
    return;
  }
  const uint32_t mant = b >> 23 ? (b & 0x7fffffu) | 0x800000u : b;
  float whole, part;
  Weigher::log2_of(mant, table, whole, part);
  whole += (float)((b >> 23 ? (int)(b >> 23) : 1) - 150);
  constexpr float kLn2 = 0.69314718055994531f, kLn2Low = (float)(0.69314718055994531 - (double)kLn2);
  const float h = __fmul_rn(kLn2, t), l = __fmaf_rn(kLn2, t, -h) + __fmul_rn(kLn2Low, t);    // ln 2 * t
  const float p = __fmul_rn(whole, h);
  const float q = __fadd_rn(__fmaf_rn(whole, h, -p), __fmaf_rn(whole, l, __fmul_rn(part, h)));
  hi = __fadd_rn(p, q);
  lo = __fsub_rn(q, __fsub_rn(hi, p));
}

// Floats as integers of the same order (both zeros alike), and back.
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

}  // namespace tq
