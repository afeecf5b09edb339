// tq_attn.cuh -- internals of the operators between the query/key/value
// product and the output product: norm and rotation of heads, append to the
// paged cache, paged attention. Nothing here is visible outside the library.
#pragma once

#include <cuda_bf16.h>

#include "tq_internal.cuh"

namespace tq {

// Status word value (beside kDevOk, kDevTimeout): a page, sequence or length
// out of range.
constexpr int kDevIndex = 2;

// Records for the stream that a kernel other than the matmuls was enqueued, so
// that the next matmul waits before it reads.
void note_other_kernel(cudaStream_t s);
cudaError_t status_word(int** out);

constexpr int kMaxRopeDim = 256;   // largest head of tq_qk_norm_rope
constexpr int kMaxPositions = 1 << 30;   // of a sequence, and rows of a head of an attention call
constexpr int kMaxKvDim = 128;     // largest head of the paged cache

// One of the inputs of the norm/rotation kernel: its heads, where they come
// from and where they go.
struct HeadSet {
  const void* x;
  void* y;              // direct output (null: into the cache, or nothing)
  const float* w;       // norm weight or null
  int64_t x_stride, y_stride;
  int heads;
  int rotate;           // 0: values, converted only
};

struct RopeCall {
  HeadSet set[3];       // q, k, v
  int x_type, y_type;
  int head_dim, half;   // half = rot_dim / 2
  int interleaved;
  float amplitude, eps;
  const uint64_t* turns;
  const int32_t* positions;
  int64_t ntok;
  // append: k and v (sets 1, 2) go to the cache
  int append;
  const int32_t* seq_ids;
  tq_paged_kv kv;
  int* status;
};

cudaError_t launch_norm_rope(const RopeCall& c, cudaStream_t s);

constexpr int kMaxSplits = 128;    // key ranges of a row tile
constexpr int kMaxCluster = 8;     // of which so many can be one cluster

// How a paged attention call is cut: a function of its sizes alone, so that
// the workspace size is too.
struct AttnPlan {
  bool chunk;           // the kernel for many rows
  int tile_rows;        // rows (token, query head) of a row tile
  int key_tile;         // keys of a tile
  int64_t tiles_x;      // row tiles: of a sequence (few rows), numbers for all (many)
  int nsplit;           // few rows: key ranges of a row tile,
  int chunk_tiles;      // and key tiles of a range,
  int cluster;          // and ranges that join in a cluster (1: none)
  int blocks;           // many rows: thread blocks
  int64_t part_rows;    // rows of partial results
  int64_t ws_bytes;
};
AttnPlan attn_plan(int64_t nseq, int64_t ntok, int64_t q_heads, int64_t kv_heads,
                   int64_t head_dim, int64_t max_q, int64_t max_kv, int64_t window);

struct AttnCall {
  const void* q;
  int64_t q_stride;
  tq_paged_kv kv;
  const int32_t* q_start;
  const int32_t* kv_len;
  void* o;
  int64_t o_stride;
  int o_type;
  float* lse;
  int64_t ntok, q_heads, max_q, max_kv;
  float scale;
  int64_t window;
  // partial results: few rows [nsplit][ntok][q_heads] rows (nsplit > 1), many
  // rows two row tiles a block
  float* part_o;        // [part_rows][head_dim]
  float* part_lse;      // [part_rows], base-2 logarithms
  void* cuts;
  int* status;
  AttnPlan plan;
};

cudaError_t launch_attention(const AttnCall& c, cudaStream_t s);

// ---------------------------------------------------------------- conversions

template <typename T> struct Elem;
template <> struct Elem<float> {
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};

template <typename T, int N> struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

}  // namespace tq
