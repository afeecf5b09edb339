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
// a rotation needs no exchange and the norm one shuffle sum. A group takes
// HEADS heads of one token and issues all their loads before it uses any. The
// sines and cosines of a block's tokens are computed once for all its groups,
// into shared memory, while those loads are under way (by every group for
// itself they were half of the instructions, and those the limit: 77 us for
// 8192 tokens of 48 heads of 128, where the bytes take 44). A block serves one
// of the sets (queries, keys, values), so that nothing but the data differs
// between its threads.
#include <cmath>
#include <cstring>

#include "tq_attn.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;

template <typename T, int N>
__device__ __forceinline__ void store_vec(T* y, const float (&x)[N]) {
  Vec<T, N> v;
#pragma unroll
  for (int e = 0; e < N; ++e) v.v[e] = Elem<T>::down(x[e]);
  *reinterpret_cast<Vec<T, N>*>(y) = v;
}

struct Cut {            // how the sets are dealt to blocks
  int lanes;            // of a group, a power of two
  int first[4];         // first block of each set, and the end
  int chunks[3];        // groups of a token
};

template <typename TI, typename TO, int VEC, int NU, int HEADS>
__global__ void __launch_bounds__(kThreads, 4)
norm_rope_kernel(const __grid_constant__ RopeCall c, const __grid_constant__ Cut cut) {
  // (cos, sin) of the block's tokens: groups * pairs of a head at most, which
  // is kThreads * NU * VEC
  __shared__ float2 turn[kThreads * NU * VEC];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int k = blockIdx.x < cut.first[1] ? 0 : blockIdx.x < cut.first[2] ? 1 : 2;
  const HeadSet& hs = c.set[k];
  const int lanes = cut.lanes, chunks = cut.chunks[k];
  const int groups = kThreads / lanes;
  const int64_t items = c.ntok * chunks;
  const int64_t item0 = (int64_t)(blockIdx.x - cut.first[k]) * groups;
  // groups past the end shadow the last one up to their stores: the shuffles
  // below want whole warps
  const int64_t mine = item0 + threadIdx.x / lanes;
  const bool live = mine < items;
  auto token_of = [&](int64_t i) {
    return items <= 0x7fffffff ? (int64_t)((uint32_t)i / (uint32_t)chunks) : i / chunks;
  };
  const int64_t it = live ? mine : items - 1;
  const int64_t tok = token_of(it), tok0 = token_of(item0);
  const int first = (int)(it - tok * chunks);
  const int lane = threadIdx.x & (lanes - 1);
  const int units = c.head_dim / (2 * VEC), runits = hs.rotate ? c.half / VEC : 0;

  // this lane's pairs: where their two vectors start in a head
  int o0[NU], o1[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = lane + i * lanes;
    o0[i] = 2 * u * VEC;
    o1[i] = o0[i] + VEC;
    if (u < runits && !c.interleaved) {
      o0[i] = u * VEC;
      o1[i] = c.half + u * VEC;
    }
  }

  // the group's heads: first, first + chunks, ...
  Vec<TI, VEC> xa[HEADS][NU], xb[HEADS][NU];
  const TI* x = static_cast<const TI*>(hs.x) + tok * hs.x_stride + first * c.head_dim;
#pragma unroll
  for (int j = 0; j < HEADS; ++j)
    if (first + j * chunks < hs.heads) {
#pragma unroll
      for (int i = 0; i < NU; ++i)
        if (lane + i * lanes < units) {
          xa[j][i] = *reinterpret_cast<const Vec<TI, VEC>*>(x + j * chunks * c.head_dim + o0[i]);
          xb[j][i] = *reinterpret_cast<const Vec<TI, VEC>*>(x + j * chunks * c.head_dim + o1[i]);
        }
    }

  if (runits > 0) {
    const int n = ((int)(token_of(min(item0 + groups, items) - 1) - tok0) + 1) * c.half;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int t = i / c.half;
      const int pos = c.positions[tok0 + t];
      // the upper half of the 64-bit fraction, a signed 32-bit one of a turn
      const uint64_t frac = (uint64_t)(int64_t)pos * c.turns[i - t * c.half];
      float s, co;
      sincospif((float)(int32_t)(frac >> 32) * 0x1p-31f, &s, &co);
      turn[i] = make_float2(co * c.amplitude, s * c.amplitude);
    }
    __syncthreads();
  }

  // where the token goes in the cache
  int64_t slot = -1;
  bool write = live;
  if (c.append) {
    const int pos = c.positions[tok];
    if (pos < 0) {
      write = false;   // padding
    } else if (k > 0) {
      const int seq = c.seq_ids[tok];
      const int lp = pos / (int)c.kv.page_size;
      int page = -1;
      if (seq >= 0 && seq < c.kv.nseq && lp < c.kv.table_width)
        page = c.kv.block_table[seq * c.kv.table_stride + lp];
      if (page >= 0 && page < c.kv.pages) {
        slot = page * c.kv.page_stride + (pos - lp * (int)c.kv.page_size) * c.kv.slot_stride;
      } else {
        if (lane == 0 && live) *c.status = kDevIndex;
        write = false;
      }
    }
  }
  TO* y = hs.y ? static_cast<TO*>(hs.y) + tok * hs.y_stride
               : static_cast<TO*>(k == 1 ? c.kv.k : c.kv.v) + slot;
  const int64_t y_head = hs.y ? c.head_dim : c.kv.head_stride;

  float wa[NU][VEC], wb[NU][VEC];
  if (hs.w) {
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const bool have = lane + i * lanes < units;
        wa[i][e] = have ? __ldg(hs.w + o0[i] + e) : 0.0f;
        wb[i][e] = have ? __ldg(hs.w + o1[i] + e) : 0.0f;
      }
  }
  const float2* const cs = turn + (tok - tok0) * c.half;

#pragma unroll
  for (int j = 0; j < HEADS; ++j) {
    const int head = first + j * chunks;
    const bool there = head < hs.heads;
    float a[NU][VEC], b[NU][VEC], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const bool have = there && lane + i * lanes < units;
        a[i][e] = have ? Elem<TI>::up(xa[j][i].v[e]) : 0.0f;
        b[i][e] = have ? Elem<TI>::up(xb[j][i].v[e]) : 0.0f;
        sum = fmaf(a[i][e], a[i][e], fmaf(b[i][e], b[i][e], sum));
      }
    if (hs.w) {
      for (int d = lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const float r = rsqrtf(sum / (float)c.head_dim + c.eps);
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          a[i][e] *= r * wa[i][e];
          b[i][e] *= r * wb[i][e];
        }
    }
    if (!there || !write) continue;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = lane + i * lanes;
      if (u >= units) continue;
      if (u < runits) {
        if (!c.interleaved) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float2 t = cs[u * VEC + e];
            const float p = a[i][e], q = b[i][e];
            a[i][e] = p * t.x - q * t.y;
            b[i][e] = q * t.x + p * t.y;
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
            const float2 t = cs[u * VEC + n];
            const float p = z[2 * n], q = z[2 * n + 1];
            z[2 * n] = p * t.x - q * t.y;
            z[2 * n + 1] = q * t.x + p * t.y;
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            a[i][e] = z[e];
            b[i][e] = z[VEC + e];
          }
        }
      }
      store_vec<TO, VEC>(y + head * y_head + o0[i], a[i]);
      store_vec<TO, VEC>(y + head * y_head + o1[i], b[i]);
    }
  }
}

template <typename TI, typename TO, int VEC, int NU, int HEADS>
cudaError_t launch_as(const RopeCall& c, cudaStream_t s) {
  const int units = c.head_dim / (2 * VEC);
  Cut cut = {};
  cut.lanes = 1;
  while (cut.lanes < 32 && cut.lanes < units) cut.lanes *= 2;
  const int groups = kThreads / cut.lanes;
  int64_t grid = 0;
  for (int k = 0; k < 3; ++k) {
    cut.first[k] = (int)grid;
    cut.chunks[k] = (c.set[k].heads + HEADS - 1) / HEADS;
    grid += (c.ntok * cut.chunks[k] + groups - 1) / groups;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  }
  cut.first[3] = (int)grid;
  return launch_pdl(norm_rope_kernel<TI, TO, VEC, NU, HEADS>, dim3((unsigned)grid),
                    dim3(kThreads), 0, s, c, cut);
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
      // one head a group where heads are few, so that all SMs get some
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
