// tq_attn_dev.cuh -- what the two attention kernels and the join of their
// partial results share: parameters, TMA boxes of the paged cache, stores.
#pragma once

#include <cuda.h>

#include "tq_attn.cuh"
#include "tq_ring.cuh"

namespace tq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kWaitNs = 1000000000ull;   // limit of the waits in the attention kernels

struct AttnParams {
  const void* q;
  void* o;
  float* lse;
  float* part_o;
  float* part_lse;
  void* cuts;           // many rows: the row tiles that were cut, one entry a block
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t q_stride, o_stride, table_stride, table_width;
  int64_t ntok;
  int* status;
  uint64_t stall_ns;    // test facility, if not 0: the first block requests no tiles,
                        // and its waits have this limit
  uint32_t group_inv;   // ceil(2^32 / group), exact for numbers below 2^16; 0: divide
  int q_heads, group, dim, page_size, pages, box_rows;
  int nseq, tiles_x, nsplit, chunk_tiles, max_q;
  int cluster;          // few rows: splits that join within a cluster (1: none)
  int o_type;
  int window;           // 0: none
  int max_positions;    // of the block table; a longer kv_len counts as this
  float scale_log2;
};

// The weights of the keys are rounded to T for their product with the values,
// which the tensor cores want alike; their sum, the divisor, takes them in 32
// bits. In f16, where the largest weight were 1, those below 2^-25 would vanish
// from the product and stay in the sum (20,000 keys with a score 18 below one
// key's came out as nothing), so weights are 2^Up times that, up to 2^15 of the
// 2^16 that f16 holds: smaller ones keep all bits to 2^-14 - Up. The power is
// taken off the maximum at the end. bf16 has the exponents of 32 bits.
template <typename T, int Up> struct Scaled { static constexpr float kUp = 0.0f; };
template <int Up> struct Scaled<__half, Up> { static constexpr float kUp = Up; };
// The exponent's addend for the reference m of a row (finite or 0).
template <typename T, int Up> __device__ __forceinline__ float addend(float m) {
  return Scaled<T, Up>::kUp != 0.0f ? Scaled<T, Up>::kUp - m : -m;
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 4-D tiled TMA load {64 values, box_rows slots, 1 head, 1 page}.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int slot,
                                        int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// Byte offset of 16-byte chunk j of row r in a 64-value-wide tile of 128-byte
// rows with the 128-byte swizzle (tile 1024-byte aligned).
__device__ __forceinline__ uint32_t swz(int r, int j) {
  return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4));
}

__device__ __forceinline__ void store_out(void* o, int type, int64_t at, float x) {
  if (type == TQ_F32) static_cast<float*>(o)[at] = x;
  else if (type == TQ_F16) static_cast<__half*>(o)[at] = __float2half_rn(x);
  else static_cast<__nv_bfloat16*>(o)[at] = __float2bfloat16_rn(x);
}

// Four consecutive values from a multiple of 4 on: one store where the address
// allows it.
__device__ __forceinline__ void store_out4(void* o, int type, int64_t at, const float (&x)[4]) {
  if (type == TQ_F32) {
    float* y = static_cast<float*>(o) + at;
    if (((uintptr_t)y & 15u) == 0) {
      *reinterpret_cast<float4*>(y) = make_float4(x[0], x[1], x[2], x[3]);
      return;
    }
  } else {
    uint16_t* y = static_cast<uint16_t*>(o) + at;
    if (((uintptr_t)y & 7u) == 0) {
      *reinterpret_cast<uint2*>(y) =
          type == TQ_F16
              ? make_uint2(pack2<__half>(x[0], x[1]), pack2<__half>(x[2], x[3]))
              : make_uint2(pack2<__nv_bfloat16>(x[0], x[1]), pack2<__nv_bfloat16>(x[2], x[3]));
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) store_out(o, type, at + e, x[e]);
}

// The first n (a multiple of 8, at least 8) of 16 consecutive values: whole
// 32-byte sectors a store where the address allows it.
__device__ __forceinline__ void store32(void* y, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"l"(y), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
               "r"(w[7]) : "memory");
}
__device__ __forceinline__ void store_out16(void* o, int type, int64_t at, const float (&x)[16], int n) {
  char* const y = static_cast<char*>(o) + at * (type == TQ_F32 ? 4 : 2);
  if (n >= 16 && ((uintptr_t)y & 31u) == 0) {
    uint32_t w[8];
    if (type == TQ_F32) {
#pragma unroll
      for (int c = 0; c < 16; c += 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(x[c + e]);
        store32(y + c * 4, w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = type == TQ_F16 ? pack2<__half>(x[2 * e], x[2 * e + 1])
                              : pack2<__nv_bfloat16>(x[2 * e], x[2 * e + 1]);
      store32(y, w);
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    const float v[4] = {x[c], x[c + 1], x[c + 2], x[c + 3]};
    if (c < n) store_out4(o, type, at + c, v);
  }
}

cudaError_t launch_attn_decode(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, cudaStream_t s);
cudaError_t launch_attn_chunk(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                              const CUtensorMap& vmap, cudaStream_t s);

}  // namespace tq
