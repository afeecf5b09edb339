// tq_rope.cu -- the launch of the norm/rotation kernel by input type, and the
// frequency tables on the host.
#include <cmath>

#include "tq_attn.cuh"

namespace tq {

cudaError_t launch_norm_rope_f32(const RopeCall& c, cudaStream_t s);
cudaError_t launch_norm_rope_f16(const RopeCall& c, cudaStream_t s);
cudaError_t launch_norm_rope_bf16(const RopeCall& c, cudaStream_t s);

cudaError_t launch_norm_rope(const RopeCall& c, cudaStream_t s) {
  switch (c.x_type) {
    case TQ_F32: return launch_norm_rope_f32(c, s);
    case TQ_F16: return launch_norm_rope_f16(c, s);
    default: return launch_norm_rope_bf16(c, s);
  }
}

}  // namespace tq

extern "C" int tq_rope_turns(int64_t rot_dim, double base, int kind, double factor,
                             double original_len, double low, double high, uint64_t* turns,
                             float* amplitude) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (rot_dim < 0 || rot_dim % 2 != 0 || !(base > 0) || !std::isfinite(base) ||
      kind < TQ_ROPE_PLAIN || kind > TQ_ROPE_BANDS)
    return TQ_ERR_SHAPE;
  if (kind != TQ_ROPE_PLAIN && !(factor >= 1 && std::isfinite(factor))) return TQ_ERR_SHAPE;
  if (kind == TQ_ROPE_BASE && rot_dim == 2) return TQ_ERR_SHAPE;
  const bool banded = kind == TQ_ROPE_RAMP || kind == TQ_ROPE_BANDS;
  if (banded && !(original_len > 0 && low > 0 && low < high && std::isfinite(original_len) &&
                  std::isfinite(high)))
    return TQ_ERR_SHAPE;
  if (kind == TQ_ROPE_RAMP && !(base > 1)) return TQ_ERR_SHAPE;
  if (rot_dim > 0 && !turns) return TQ_ERR_NULL;
  if (amplitude) *amplitude = kind == TQ_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  if (kind == TQ_ROPE_BASE && rot_dim > 2)
    base *= std::pow(factor, (double)rot_dim / (double)(rot_dim - 2));
  // the ramp: pairs up to `kept` make `high` turns or more, those from `divided`
  // on `low` or fewer (either may lie past the table, at one end or the other)
  double kept = 0, divided = 0;
  if (kind == TQ_ROPE_RAMP) {
    // the pair index at which a pair makes n turns over original_len positions
    auto index = [&](double n) {
      return 0.5 * rot_dim * std::log(original_len / (n * kTwoPi)) / std::log(base);
    };
    kept = std::floor(index(high));
    divided = std::ceil(index(low));
  }
  for (int64_t i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * (double)i / (double)rot_dim);
    double keep = 1.0;
    if (kind == TQ_ROPE_LINEAR) keep = 0.0;
    if (kind == TQ_ROPE_RAMP) {
      const double first = std::fmax(kept, 0.0), last = std::fmin(divided, (double)(rot_dim - 1));
      keep = (double)i <= kept ? 1.0 : (double)i >= divided ? 0.0 : 1.0 - ((double)i - first) / (last - first);
    }
    if (kind == TQ_ROPE_BANDS)
      keep = std::fmin(std::fmax((original_len * f / kTwoPi - low) / (high - low), 0.0), 1.0);
    if (keep < 1.0) f = f * keep + f / factor * (1.0 - keep);
    // the fraction of a turn, rounded to 64 bits (the product by 2^64 is exact)
    double t = f / kTwoPi;
    t -= std::floor(t);
    const double scaled = std::nearbyint(std::ldexp(t, 64));
    turns[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
  }
  return TQ_OK;
}
