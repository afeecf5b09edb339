// tq_rope.cu -- norm and rotation of query and key heads, and their append to
// the paged cache with the values, in one pass; the frequency tables on the host.
//
// For a head x of D values: r = 1 / sqrt(mean(x^2) + eps), x' = x r w, then
// (a, b) -> m (a cos - b sin, b cos + a sin) for the pairs of the first
// rot_dim values. The angle is position * turns mod 2^64, a 64-bit fraction of
// a turn: exact integer arithmetic drops whole turns, and sincospif takes the
// rest.
//
// Bound by the bytes of the heads, read once and written once. A group of
// lanes holds whole heads in registers: a lane owns `VEC` pairs (two vectors
// of VEC values, at i and i + rot_dim/2, or side by side when interleaved), so
// a rotation needs no exchange and the norm one shuffle sum. The lane's pairs
// are the same in every head, so one sine and cosine per pair serves the
// group's RPG heads of a token; their loads are all issued before any is used.
#include <cmath>
#include <cstring>

#include "tq_attn.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;

template <typename TI, typename TO, int VEC, int NU, int RPG>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(const __grid_constant__ RopeCall c, int lanes, int rows, int chunks,
                 int64_t items) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t item = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  // groups past the end shadow the last one up to their stores: the shuffles
  // below want whole warps
  const bool live = item < items;
  const int64_t it = live ? item : items - 1;
  const int64_t tok =
      items <= 0x7fffffff ? (int64_t)((uint32_t)it / (uint32_t)chunks) : it / chunks;
  const int first = (int)(it - tok * chunks);
  const int lane = threadIdx.x & (lanes - 1);
  const int units = c.head_dim / (2 * VEC), runits = c.half / VEC;

  // this lane's pairs: where their two vectors start in a head, and whether
  // they are rotated
  int o0[NU], o1[NU];
  bool have[NU], rot[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = lane + i * lanes;
    have[i] = u < units;
    rot[i] = u < runits;
    o0[i] = 2 * u * VEC;
    o1[i] = o0[i] + VEC;
    if (rot[i] && !c.interleaved) {
      o0[i] = u * VEC;
      o1[i] = c.half + u * VEC;
    }
  }

  // loads of all heads of the group
  Vec<TI, VEC> xa[RPG][NU], xb[RPG][NU];
  int set[RPG], head[RPG];
#pragma unroll
  for (int j = 0; j < RPG; ++j) {
    int r = first + j * chunks;
    set[j] = -1;
    head[j] = 0;
    if (r < rows) {
      int k = 0;
      if (r >= c.set[0].heads) {
        r -= c.set[0].heads;
        k = 1;
        if (r >= c.set[1].heads) {
          r -= c.set[1].heads;
          k = 2;
        }
      }
      set[j] = k;
      head[j] = r;
      const TI* x = static_cast<const TI*>(c.set[k].x) + tok * c.set[k].x_stride +
                    (int64_t)r * c.head_dim;
#pragma unroll
      for (int i = 0; i < NU; ++i)
        if (have[i]) {
          xa[j][i] = *reinterpret_cast<const Vec<TI, VEC>*>(x + o0[i]);
          xb[j][i] = *reinterpret_cast<const Vec<TI, VEC>*>(x + o1[i]);
        }
    }
  }

  const int pos = c.positions ? c.positions[tok] : 0;
  float cs[NU][VEC], sn[NU][VEC];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      cs[i][e] = 1.0f;
      sn[i][e] = 0.0f;
      if (rot[i]) {
        const uint64_t f = c.turns[(lane + i * lanes) * VEC + e];
        // signed fraction of a turn in [-1/2, 1/2); sincospif wants half turns
        const float t = (float)(int64_t)((uint64_t)(int64_t)pos * f) * 0x1p-63f;
        sincospif(t, &sn[i][e], &cs[i][e]);
        cs[i][e] *= c.amplitude;
        sn[i][e] *= c.amplitude;
      }
    }

  // where the token goes in the cache
  int64_t slot = -1;
  bool write = live;
  if (c.append) {
    if (pos < 0) {
      write = false;   // padding
    } else {
      const int seq = c.seq_ids[tok];
      const int lp = pos / (int)c.kv.page_size;
      int page = -1;
      if (seq >= 0 && seq < c.kv.nseq && lp < c.kv.table_width)
        page = c.kv.block_table[seq * c.kv.table_stride + lp];
      if (page >= 0 && page < c.kv.pages)
        slot = page * c.kv.page_stride + (pos - lp * (int)c.kv.page_size) * c.kv.slot_stride;
      else if (lane == 0 && live)
        *c.status = kDevIndex;
    }
  }

#pragma unroll
  for (int j = 0; j < RPG; ++j) {
    const int k = set[j];
    float a[NU][VEC], b[NU][VEC], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        a[i][e] = b[i][e] = 0.0f;
        if (k >= 0 && have[i]) {
          a[i][e] = Elem<TI>::up(xa[j][i].v[e]);
          b[i][e] = Elem<TI>::up(xb[j][i].v[e]);
          sum += a[i][e] * a[i][e] + b[i][e] * b[i][e];
        }
      }
    for (int d = lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (k < 0 || !write) continue;
    const HeadSet& hs = c.set[k];
    TO* y;
    if (hs.y) {
      y = static_cast<TO*>(hs.y) + tok * hs.y_stride + (int64_t)head[j] * c.head_dim;
    } else {
      if (slot < 0) continue;
      y = static_cast<TO*>(k == 1 ? c.kv.k : c.kv.v) + slot + (int64_t)head[j] * c.kv.head_stride;
    }
    const float r = hs.w ? 1.0f / sqrtf(sum / (float)c.head_dim + c.eps) : 1.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (!have[i]) continue;
      if (hs.w) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          a[i][e] = a[i][e] * r * __ldg(hs.w + o0[i] + e);
          b[i][e] = b[i][e] * r * __ldg(hs.w + o1[i] + e);
        }
      }
      if (hs.rotate && rot[i]) {
        if (!c.interleaved) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float p = a[i][e], q = b[i][e];
            a[i][e] = p * cs[i][e] - q * sn[i][e];
            b[i][e] = q * cs[i][e] + p * sn[i][e];
          }
        } else {
          // the unit's 2 VEC values are consecutive: pair n is values 2n, 2n + 1
          float z[2 * VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            z[e] = a[i][e];
            z[VEC + e] = b[i][e];
          }
#pragma unroll
          for (int n = 0; n < VEC; ++n) {
            const float p = z[2 * n], q = z[2 * n + 1];
            z[2 * n] = p * cs[i][n] - q * sn[i][n];
            z[2 * n + 1] = q * cs[i][n] + p * sn[i][n];
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            a[i][e] = z[e];
            b[i][e] = z[VEC + e];
          }
        }
      }
      Vec<TO, VEC> ya, yb;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        ya.v[e] = Elem<TO>::down(a[i][e]);
        yb.v[e] = Elem<TO>::down(b[i][e]);
      }
      *reinterpret_cast<Vec<TO, VEC>*>(y + o0[i]) = ya;
      *reinterpret_cast<Vec<TO, VEC>*>(y + o1[i]) = yb;
    }
  }
}

template <typename TI, typename TO, int VEC, int NU, int RPG>
cudaError_t launch_as(const RopeCall& c, cudaStream_t s) {
  const int units = c.head_dim / (2 * VEC);
  int lanes = 1;
  while (lanes < 32 && lanes < units) lanes *= 2;
  const int rows = c.set[0].heads + c.set[1].heads + c.set[2].heads;
  const int chunks = (rows + RPG - 1) / RPG;
  const int64_t items = c.ntok * chunks;
  const int per_cta = kThreads / lanes;
  const int64_t grid = (items + per_cta - 1) / per_cta;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(norm_rope_kernel<TI, TO, VEC, NU, RPG>, dim3((unsigned)grid), dim3(kThreads),
                    0, s, c, lanes, rows, chunks, items);
}

// Widest vectors that the sizes, strides and addresses allow.
int vector_width(const RopeCall& c) {
  const int64_t in = c.x_type == TQ_F32 ? 4 : 2, out = c.y_type == TQ_F32 ? 4 : 2;
  for (int v = 4; v > 1; v /= 2) {
    bool ok = c.half % v == 0 && (c.head_dim - 2 * c.half) % (2 * v) == 0;
    for (int k = 0; k < 3 && ok; ++k) {
      const HeadSet& h = c.set[k];
      if (!h.heads) continue;
      ok = c.head_dim % v == 0 && h.x_stride % v == 0 && (uintptr_t)h.x % (in * v) == 0;
      if (ok && h.y) ok = h.y_stride % v == 0 && (uintptr_t)h.y % (out * v) == 0;
    }
    if (ok) return v;
  }
  return 1;
}

template <typename TI, typename TO>
cudaError_t launch_types(const RopeCall& c, cudaStream_t s) {
  const int64_t rows = c.set[0].heads + c.set[1].heads + c.set[2].heads;
  switch (vector_width(c)) {
    case 4:
      // one head per group where heads are few, so that all SMs get some
      if (c.ntok * rows < 8192) return launch_as<TI, TO, 4, 1, 1>(c, s);
      return launch_as<TI, TO, 4, 1, 4>(c, s);
    case 2: return launch_as<TI, TO, 2, 2, 2>(c, s);
    default: return launch_as<TI, TO, 1, 4, 1>(c, s);
  }
}

template <typename TI>
cudaError_t launch_out(const RopeCall& c, cudaStream_t s) {
  switch (c.y_type) {
    case TQ_F32: return launch_types<TI, float>(c, s);
    case TQ_F16: return launch_types<TI, __half>(c, s);
    default: return launch_types<TI, __nv_bfloat16>(c, s);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const RopeCall& c, cudaStream_t s) {
  switch (c.x_type) {
    case TQ_F32: return launch_out<float>(c, s);
    case TQ_F16: return launch_out<__half>(c, s);
    default: return launch_out<__nv_bfloat16>(c, s);
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
  double first = 0, last = 0;
  if (kind == TQ_ROPE_RAMP) {
    // the pair index at which a pair makes n turns over original_len positions
    auto index = [&](double n) {
      return 0.5 * rot_dim * std::log(original_len / (n * kTwoPi)) / std::log(base);
    };
    first = std::fmax(std::floor(index(high)), 0.0);
    last = std::fmin(std::ceil(index(low)), (double)(rot_dim - 1));
    if (first == last) last += 0.001;
  }
  for (int64_t i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * (double)i / (double)rot_dim);
    double keep = 1.0;
    if (kind == TQ_ROPE_LINEAR) keep = 0.0;
    if (kind == TQ_ROPE_RAMP)
      keep = 1.0 - std::fmin(std::fmax(((double)i - first) / (last - first), 0.0), 1.0);
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
