// tq_rope.cuh -- norm and rotation of query and key heads, and their append to
// the paged cache with the values, in one pass.
//
// For a head x of D values: r = 1 / sqrt(mean(x^2) + eps), x' = x r w, then
// (a, b) -> m (a cos - b sin, b cos + a sin) for the pairs of the first
// rot_dim values. The angle is position * turns mod 2^64, a 64-bit fraction of
// a turn: exact integer arithmetic drops whole turns, and sincospif takes the
// rest.
//
// Bound by the bytes of the heads, read once and written once, with f32 input
// (8192 tokens of 48 heads of 128 to bf16: 53 us where the bytes take 45). With
// 16-bit input the bytes are two thirds, the instructions are not (bf16 to bf16
// 50 us, f16 to f16 45, where the bytes take 30): 2.6 of 4 instructions a cycle,
// most of them conversions and the scalar arithmetic of norm and rotation. A group of
// lanes holds whole heads in registers: a lane owns `VEC` pairs (two vectors
// of VEC values, at i and i + rot_dim/2, or side by side when interleaved), so
// a rotation needs no exchange and the norm one shuffle sum. A group takes up
// to 8 heads of one token and issues the loads of four before it uses any. The
// sines and cosines of a block's tokens are computed once for all its groups,
// into shared memory, while those loads are under way (by every group for
// itself they were half of the instructions: 77 us for the f32 case). A block serves one
// of the sets (queries, keys, values), so that nothing but the data differs
// between its threads.
#pragma once

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
  int first[4];         // first block of each set, and the end
  int chunks[3];        // groups of a token
  float inv_dim;
};

template <typename TI, typename TO, int VEC, int NU, int LANES, int HEADS>
__global__ void __launch_bounds__(kThreads, 4)
norm_rope_kernel(const __grid_constant__ RopeCall c, const __grid_constant__ Cut cut) {
  constexpr int kGroups = kThreads / LANES;
  constexpr int kBatch = HEADS < 4 ? HEADS : 4;   // heads whose loads are issued together
  // (cos, sin) of the block's tokens: groups * pairs of a head at most
  __shared__ float2 turn[kThreads * NU * VEC];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int k = blockIdx.x < cut.first[1] ? 0 : blockIdx.x < cut.first[2] ? 1 : 2;
  const HeadSet& hs = c.set[k];
  const int chunks = cut.chunks[k];
  const int64_t items = c.ntok * chunks;
  const int64_t item0 = (int64_t)(blockIdx.x - cut.first[k]) * kGroups;
  // groups past the end shadow the last one up to their stores: the shuffles
  // below want whole warps
  const int64_t mine = item0 + threadIdx.x / LANES;
  const bool live = mine < items;
  auto token_of = [&](int64_t i) {
    return items <= 0x7fffffff ? (int64_t)((uint32_t)i / (uint32_t)chunks) : i / chunks;
  };
  const int64_t it = live ? mine : items - 1;
  const int64_t tok = token_of(it), tok0 = token_of(item0);
  const int first = (int)(it - tok * chunks);
  const int lane = threadIdx.x & (LANES - 1);
  const int units = c.head_dim / (2 * VEC), runits = hs.rotate ? c.half / VEC : 0;

  // this lane's pairs: where their two vectors start in a head (of lanes past
  // the head, at its start)
  int o0[NU], o1[NU];
  bool have[NU], rot[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = lane + i * LANES;
    have[i] = u < units;
    rot[i] = u < runits;
    o0[i] = have[i] ? 2 * u * VEC : 0;
    o1[i] = o0[i] + VEC;
    if (rot[i] && !c.interleaved) {
      o0[i] = u * VEC;
      o1[i] = c.half + u * VEC;
    }
  }

  // the group's heads: first, first + chunks, ..., a batch at a time; past the
  // last one that one again, up to the store
  const TI* const x = static_cast<const TI*>(hs.x) + tok * hs.x_stride;
  Vec<TI, VEC> xa[kBatch][NU], xb[kBatch][NU];
  auto load = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const TI* const xh = x + min(first + (j0 + j) * chunks, hs.heads - 1) * c.head_dim;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        xa[j][i] = *reinterpret_cast<const Vec<TI, VEC>*>(xh + o0[i]);
        xb[j][i] = *reinterpret_cast<const Vec<TI, VEC>*>(xh + o1[i]);
      }
    }
  };
  load(0);

  if (runits > 0) {
    const int n = ((int)(token_of(min(item0 + kGroups, items) - 1) - tok0) + 1) * c.half;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int t = i / c.half;
      const int pos = c.positions[tok0 + t];
      // the upper half of the 64-bit fraction, a signed 32-bit one of a turn
      const uint64_t frac = (uint64_t)(int64_t)pos * c.turns[i - t * c.half];
      float s, co;
      sincospif((float)(int32_t)(frac >> 32) * 0x1p-31f, &s, &co);
      turn[i] = make_float2(co * c.amplitude, s * c.amplitude);
    }
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
  const int64_t y_head = hs.y ? c.head_dim : c.kv.head_stride;
  TO* const y = hs.y ? static_cast<TO*>(hs.y) + tok * hs.y_stride
                     : static_cast<TO*>(k == 1 ? c.kv.k : c.kv.v) + slot;

  float wa[NU][VEC], wb[NU][VEC];
  if (hs.w) {
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        wa[i][e] = have[i] ? __ldg(hs.w + o0[i] + e) : 0.0f;
        wb[i][e] = have[i] ? __ldg(hs.w + o1[i] + e) : 0.0f;
      }
  }
  if (runits > 0) __syncthreads();
  float2 cs[NU][VEC];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      cs[i][e] = rot[i] ? turn[(int)(tok - tok0) * c.half + (lane + i * LANES) * VEC + e]
                        : make_float2(1.0f, 0.0f);

#pragma unroll 1
  for (int j0 = 0; j0 < HEADS; j0 += kBatch) {
    if (j0 > 0) load(j0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int head = first + (j0 + j) * chunks;
      float a[NU][VEC], b[NU][VEC];
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          a[i][e] = Elem<TI>::up(xa[j][i].v[e]);
          b[i][e] = Elem<TI>::up(xb[j][i].v[e]);
        }
      if (hs.w) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          float part = 0.0f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) part = fmaf(a[i][e], a[i][e], fmaf(b[i][e], b[i][e], part));
          sum += have[i] ? part : 0.0f;
        }
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float r = rsqrtf(fmaf(sum, cut.inv_dim, c.eps));
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            a[i][e] *= r * wa[i][e];
            b[i][e] *= r * wb[i][e];
          }
      }
      if (head >= hs.heads || !write) continue;
      TO* const yh = y + head * y_head;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (!have[i]) continue;
        if (rot[i]) {
          if (!c.interleaved) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float p = a[i][e], q = b[i][e];
              a[i][e] = p * cs[i][e].x - q * cs[i][e].y;
              b[i][e] = q * cs[i][e].x + p * cs[i][e].y;
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
              z[2 * n] = p * cs[i][n].x - q * cs[i][n].y;
              z[2 * n + 1] = q * cs[i][n].x + p * cs[i][n].y;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              a[i][e] = z[e];
              b[i][e] = z[VEC + e];
            }
          }
        }
        store_vec<TO, VEC>(yh + o0[i], a[i]);
        store_vec<TO, VEC>(yh + o1[i], b[i]);
      }
    }
  }
}

template <typename TI, typename TO, int VEC, int NU, int LANES, int HEADS>
cudaError_t launch_as(const RopeCall& c, cudaStream_t s) {
  constexpr int kGroups = kThreads / LANES;
  Cut cut = {};
  cut.inv_dim = 1.0f / (float)c.head_dim;
  int64_t grid = 0;
  for (int k = 0; k < 3; ++k) {
    cut.first[k] = (int)grid;
    cut.chunks[k] = (c.set[k].heads + HEADS - 1) / HEADS;
    grid += (c.ntok * cut.chunks[k] + kGroups - 1) / kGroups;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  }
  cut.first[3] = (int)grid;
  return launch_pdl(norm_rope_kernel<TI, TO, VEC, NU, LANES, HEADS>, dim3((unsigned)grid),
                    dim3(kThreads), 0, s, c, cut);
}

// One head a group where heads are few, so that all SMs get some (200 tokens of
// 48 heads 3.1 us, 5.8 with 8 a group), else up to 8, which share more (800
// tokens 7.1 us, 9.0 with one; the two are even near 24,000 heads).
template <typename TI, typename TO, int LANES>
cudaError_t launch_wide(const RopeCall& c, cudaStream_t s) {
  const int64_t rows = c.set[0].heads + c.set[1].heads + c.set[2].heads;
  return c.ntok * rows < 24576 ? launch_as<TI, TO, 4, 1, LANES, 1>(c, s)
                              : launch_as<TI, TO, 4, 1, LANES, 8>(c, s);
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
  switch (vector_width(c)) {
    case 4:
      if (c.head_dim <= 64) return launch_wide<TI, TO, 8>(c, s);
      if (c.head_dim <= 128) return launch_wide<TI, TO, 16>(c, s);
      return launch_wide<TI, TO, 32>(c, s);
    case 2: return launch_as<TI, TO, 2, 2, 32, 1>(c, s);
    default: return launch_as<TI, TO, 1, 4, 32, 1>(c, s);
  }
}

// One instantiation per input type, each in a file of its own (they compile side by side).
template <typename TI>
cudaError_t launch_out(const RopeCall& c, cudaStream_t s) {
  switch (c.y_type) {
    case TQ_F32: return launch_types<TI, float>(c, s);
    case TQ_F16: return launch_types<TI, __half>(c, s);
    default: return launch_types<TI, __nv_bfloat16>(c, s);
  }
}

}  // namespace
}  // namespace tq
