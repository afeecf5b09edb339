// tq_lora.cuh -- what the kernels of the low-rank adapters share: arguments, conversions, loads and stores
// of activations and results, the cluster.
#pragma once

#include "tq_requests.cuh"

namespace tq {

constexpr int kLargeTile = 128;    // tokens of a tile of the kernel for many tokens

// A call's arguments, for the kernels.
struct LoraArgs {
  const void* x;
  const void* z;
  void* y;
  const int32_t* ids;
  tq_lora l;
  int64_t x_stride, z_stride, y_stride;
  int y_type;
  int ntok;
  int tile;              // tokens of a tile,
  int copy_tile;         // and of one that is only copied
  int splits;            // clusters that share the rows of a tile
  int rank_from;         // (the kernel for many tokens) ranks below are done
  int copy;              // tokens without adapter are copied (Z is not Y)
  int y_vec, z_vec;      // rows of Y, of Z in 16-byte pieces
  int b_vec, b_pairs;    // rows of B in 8-byte pieces, in 4-byte pieces
  // more than kInBlock tokens: the tiles, from the grouping kernel
  const int32_t* order;  // tokens by adapter
  const int4* tiles;     // adapter, its rank, first of order, tokens
  const int* ntiles;
  int* status;
  uint64_t stall_ns;     // (the kernel for many tokens) test facility, if not 0: the first block issues no
                         // products, its waits expire after this (tq_debug_stall_next_launch)
};

// x as a tf32 value and the rest of it, rounded to tf32: good to 2^-21. The
// first part is cut, not rounded, so that it does not overflow; an infinity
// leaves no rest.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  const float h = __uint_as_float(hi), rest = x == h ? 0.0f : x - h;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
}

// The two 16-bit values of a word as 32-bit ones.
template <typename T> __device__ __forceinline__ void widen(uint32_t w, uint32_t& a, uint32_t& b);
template <> __device__ __forceinline__ void widen<__nv_bfloat16>(uint32_t w, uint32_t& a, uint32_t& b) {
  a = w << 16;
  b = w & 0xffff0000u;
}
template <> __device__ __forceinline__ void widen<__half>(uint32_t w, uint32_t& a, uint32_t& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = __float_as_uint(f.x);
  b = __float_as_uint(f.y);
}

// Eight activations from p on: 32 or 16 bytes.
template <typename TX> struct Acts {
  uint4 v[sizeof(TX) == 4 ? 2 : 1];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (auto& q : v) q = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const TX* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(v) / sizeof(v[0])); ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  // values 2 s and 2 s + 1
  __device__ __forceinline__ void pair(int s, uint32_t& a, uint32_t& b) const {
    if constexpr (sizeof(TX) == 4) {
      const uint4 q = v[s >> 1];
      a = s & 1 ? q.z : q.x;
      b = s & 1 ? q.w : q.y;
    } else {
      const uint4 q = v[0];
      widen<TX>(s == 0 ? q.x : s == 1 ? q.y : s == 2 ? q.z : q.w, a, b);
    }
  }
};

// ---------------------------------------------------------------- infinite weights
//
// A value that is exact in tf32 has a second part of zero, whose product with an infinite weight is NaN where the
// value's own is infinite. Where the parts' products are summed apart, the second sum does not count if it is NaN.
// Where they are not, a result that is NaN is computed again from whole values, which leaves those that are NaN by
// the formula: nothing in the products' loops looks for that. (Not inlined: for weights that are not sound.)

__device__ __forceinline__ float joined(float first, float second) {
  return first + fmaxf(second, -3.402823466e38f);     // (which changes no first sum that is not finite)
}
// Four values of h of a token, from row r on, of a rank of `rank`: those that are NaN are computed again as the sums
// of n (a multiple of 8) products, up to where these are NaN. (A token that holds a NaN itself, as padding may, has
// no others: it is looked through once. 8192 such tokens of rank 32 take 1.8 ms, otherwise 7.2.)
template <typename TX, typename TW>
__device__ __noinline__ float4 dots_again(float4 h, const TX* x, const TW* a, int64_t stride, int r, int rank, int n) {
  bool sound = true;
#pragma unroll 1
  for (int k = 0; k < n && sound; k += 8)
#pragma unroll
    for (int e = 0; e < 8; ++e) sound = sound && x[k + e] == x[k + e];
  float v[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (!sound || v[e] == v[e] || r + e >= rank) continue;
    const TW* const row = a + (r + e) * stride;
    float sum = 0.0f;
#pragma unroll 1
    for (int k = 0; k < n && sum == sum; k += 8)
#pragma unroll
      for (int c = 0; c < 8; ++c) sum = __fmaf_rn(Elem<TX>::up(x[k + c]), Elem<TW>::up(row[k + c]), sum);
    v[e] = sum;
  }
  return make_float4(v[0], v[1], v[2], v[3]);
}
// One row of B times h in its two parts, value r of them at at(r), up to where the sum is NaN.
template <typename TW, typename At>
__device__ __forceinline__ float row_again(const float* hi, const float* lo, At at, const TW* b, int n) {
  float sum = 0.0f;
#pragma unroll 1
  for (int r = 0; r < n && sum == sum; ++r) sum = __fmaf_rn(hi[at(r)] + lo[at(r)], Elem<TW>::up(b[r]), sum);
  return sum;
}

// ---------------------------------------------------------------- Y and Z

__device__ __forceinline__ float up(uint16_t v, int type) {
  return type == TQ_F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ uint16_t down(float v, int type) {
  return type == TQ_F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Eight consecutive values from `at` on, at an address of a multiple of 16 bytes, as they are (w[0..7],
// or w[0..3]), and back from floats.
__device__ __forceinline__ void load8(const void* p, int type, int64_t at, uint32_t* w) {
  const uint4* q = type == TQ_F32 ? reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(p) + at)
                                  : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  const uint4 a = q[0];
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  if (type == TQ_F32) {
    const uint4 b = q[1];
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void store8(void* p, int type, int64_t at, const float (&v)[8]) {
  if (type == TQ_F32) {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = (uint32_t)down(v[2 * e], type) | (uint32_t)down(v[2 * e + 1], type) << 16;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float up1(uint32_t w, int type) {
  return type == TQ_F32 ? __uint_as_float(w) : up((uint16_t)w, type);
}

// The rows of Z of tokens without adapter as they are, to the bit: rows begin .. begin + n - 1 of `count`
// tokens.
__device__ __forceinline__ void copy_rows(const LoraArgs& p, const int* tokens, int count, int begin, int n,
                                          int threads) {
  const int tid = threadIdx.x;
  const int bytes = p.y_type == TQ_F32 ? 4 : 2, piece = p.y_vec && p.z_vec ? 16 / bytes : 1;
  const int pieces = n / piece, left = n - pieces * piece;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
  for (int i = tid; i < count * pieces; i += threads) {
    const int j = i / pieces, at = begin + (i - j * pieces) * piece;
    const int64_t to = tokens[j] * p.y_stride + at, from = tokens[j] * p.z_stride + at;
    if (piece > 1) {
      reinterpret_cast<uint4*>(static_cast<char*>(p.y) + to * bytes)[0] =
          p.z ? reinterpret_cast<const uint4*>(static_cast<const char*>(p.z) + from * bytes)[0] : zero;
    } else if (bytes == 4) {
      static_cast<uint32_t*>(p.y)[to] = p.z ? static_cast<const uint32_t*>(p.z)[from] : 0u;
    } else {
      static_cast<uint16_t*>(p.y)[to] = p.z ? static_cast<const uint16_t*>(p.z)[from] : (uint16_t)0;
    }
  }
  for (int i = tid; i < count * left; i += threads) {
    const int j = i / left, at = begin + pieces * piece + i - j * left;
    const int64_t to = tokens[j] * p.y_stride + at, from = tokens[j] * p.z_stride + at;
    if (bytes == 4) static_cast<uint32_t*>(p.y)[to] = p.z ? static_cast<const uint32_t*>(p.z)[from] : 0u;
    else static_cast<uint16_t*>(p.y)[to] = p.z ? static_cast<const uint16_t*>(p.z)[from] : (uint16_t)0;
  }
}

// ---------------------------------------------------------------- the cluster

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 load_remote(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// The kernel for many tokens of an adapter: tiles of kLargeTile tokens, `tiles` of them at most.
bool lora_large_fits(const LoraArgs& a, int64_t ntok);
cudaError_t launch_lora_large(const LoraArgs& a, int64_t tiles, int x_type, cudaStream_t s);

}  // namespace tq
