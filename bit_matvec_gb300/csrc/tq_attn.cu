// tq_attn.cu -- paged attention: the launch (parameters, maps of the cache,
// which kernel) and the join of partial results.
#include <atomic>

#include "tq_attn_dev.cuh"

namespace tq {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
static_assert(kMaxSplits <= kJoinThreads, "a thread for each split");

// Joins the partial results of the splits: o = sum_s 2^(lse_s - M) o_s /
// sum_s 2^(lse_s - M), one thread block per row of one query head; a warp
// takes every eighth split, a lane four values. All loads of a block are
// independent (walking the splits one load after another measured 70 us for
// 38 of them).
__global__ void __launch_bounds__(kJoinThreads)
attn_join_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float weight[kJoinThreads];
  __shared__ float red[2][kJoinWarps];
  __shared__ float4 part[kJoinThreads];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t rows = p.ntok * p.q_heads, row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tok = row / p.q_heads;
  float lse = -INFINITY;
  if (threadIdx.x < p.nsplit) lse = p.part_lse[threadIdx.x * rows + row];
  // tokens past the last sequence's are not written
  if (tok >= p.q_start[p.nseq]) return;
  float top = lse;
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) red[0][warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, red[0][w]);
  const float w = lse == -INFINITY ? 0.0f : exp2_approx(lse - top);
  weight[threadIdx.x] = w;
  float sum = w;
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) red[1][warp] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) sum += red[1][i];
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (lane * 4 < p.dim) {
    const float* from = p.part_o + row * p.dim + lane * 4;
#pragma unroll 4
    for (int s = warp; s < p.nsplit; s += kJoinWarps) {
      // (of a range without keys the row is zeros)
      const float4 x = *reinterpret_cast<const float4*>(from + s * rows * p.dim);
      const float f = weight[s];
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    }
  }
  part[threadIdx.x] = acc;
  __syncthreads();
  if (warp == 0 && lane * 4 < p.dim) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) {
      const float4 a = part[lane + 32 * i];
      x[0] += a.x;
      x[1] += a.y;
      x[2] += a.z;
      x[3] += a.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= inv;
    store_out4(p.o, p.o_type, tok * p.o_stride + (row - tok * p.q_heads) * p.dim + lane * 4, x);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn* out) {
  // the driver's entry point, the same for every call: host threads that come
  // first at the same time each look it up
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeFn>(f);
    known.store(fn, std::memory_order_relaxed);
  }
  *out = fn;
  return cudaSuccess;
}

// The cache as {dim, slot, head, page}, in boxes of 64 values of box_rows slots.
cudaError_t cache_map(CUtensorMap* map, const tq_paged_kv& c, void* p, int box_rows) {
  EncodeFn fn;
  const cudaError_t e = encode_fn(&fn);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size,
                              (cuuint64_t)c.heads, (cuuint64_t)c.pages};
  // a stride of a dimension of size 1 is never used, but has to be encodable
  const cuuint64_t one = (cuuint64_t)c.slot_stride * 2;
  const cuuint64_t strides[3] = {one, c.heads > 1 ? (cuuint64_t)c.head_stride * 2 : one,
                                 c.pages > 1 ? (cuuint64_t)c.page_stride * 2 : one};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1}, step[4] = {1, 1, 1, 1};
  auto encode = [&]() {
    return fn(map, c.type == TQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              4, p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r != CUDA_SUCCESS) {
    // The driver wants the device's context to be current in the calling thread.
    // A launch sees to that itself, but in a host thread whose first CUDA call
    // this is there was none yet; setting the device does it.
    int dev = 0;
    cudaError_t s = cudaGetDevice(&dev);
    if (s == cudaSuccess) s = cudaSetDevice(dev);
    if (s != cudaSuccess) return s;
    r = encode();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attention(const AttnCall& c, cudaStream_t s) {
  AttnParams p = {};
  p.q = c.q;
  p.o = c.o;
  p.lse = c.lse;
  p.part_o = c.part_o;
  p.part_lse = c.part_lse;
  p.cuts = c.cuts;
  p.q_start = c.q_start;
  p.kv_len = c.kv_len;
  p.table = c.kv.block_table;
  p.q_stride = c.q_stride;
  p.o_stride = c.o_stride;
  p.table_stride = c.kv.table_stride;
  p.table_width = c.kv.table_width;
  p.ntok = c.ntok;
  p.status = c.status;
  p.stall_ns = (uint64_t)take_debug_stall();
  p.q_heads = (int)c.q_heads;
  p.group = (int)(c.q_heads / c.kv.heads);
  // x * group < 2^32 makes the high product of x and the rounded-up reciprocal
  // x / group; row numbers of a tile are below group + 256
  if (p.group > 1 && p.group < (1 << 15))
    p.group_inv = (uint32_t)(((uint64_t(1) << 32) + p.group - 1) / p.group);
  p.dim = (int)c.kv.head_dim;
  p.page_size = (int)c.kv.page_size;
  p.pages = (int)c.kv.pages;
  // boxes are pieces of a page and of a key tile
  p.box_rows = (int)(c.kv.page_size & -c.kv.page_size);
  if (p.box_rows > c.plan.key_tile) p.box_rows = c.plan.key_tile;
  p.nseq = (int)c.kv.nseq;
  p.tiles_x = (int)c.plan.tiles_x;
  p.nsplit = c.plan.nsplit;
  p.chunk_tiles = c.plan.chunk_tiles;
  p.cluster = c.plan.cluster;
  p.max_q = (int)c.max_q;
  p.o_type = c.o_type;
  p.window = c.window >= kMaxPositions ? 0 : (int)c.window;
  const int64_t positions = c.kv.table_width * c.kv.page_size;
  p.max_positions = positions < kMaxPositions ? (int)positions : kMaxPositions;
  p.scale_log2 = c.scale * kLog2e;
  CUtensorMap kmap, vmap;
  cudaError_t e = cache_map(&kmap, c.kv, c.kv.k, p.box_rows);
  if (e == cudaSuccess) e = cache_map(&vmap, c.kv, c.kv.v, p.box_rows);
  if (e != cudaSuccess) return e;
  if (c.plan.chunk) return launch_attn_chunk(p, c, kmap, vmap, s);
  e = launch_attn_decode(p, c, kmap, vmap, s);
  if (e != cudaSuccess || p.nsplit == p.cluster) return e;
  const int64_t grid = c.ntok * c.q_heads;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(attn_join_kernel, dim3((unsigned)grid), dim3(kJoinThreads), 0, s, p);
}

}  // namespace tq
