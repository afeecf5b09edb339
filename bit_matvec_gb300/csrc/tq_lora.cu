// tq_lora.cu -- low-rank adapters of many requests beside a shared product:
// Y[t] = Z[t] + scale B (A x[t]) with the adapter of each token.
//
// One thread block per token: a warp per row of A, then a thread per output.
#include "tq_requests.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;

struct Args {
  const void* x;
  const void* z;
  void* y;
  const int32_t* ids;
  tq_lora l;
  int64_t x_stride, z_stride, y_stride;
  int x_type, y_type;
  int* status;
};

__device__ __forceinline__ float load(const void* p, int type, int64_t at) {
  if (type == TQ_F32) return static_cast<const float*>(p)[at];
  if (type == TQ_F16) return __half2float(static_cast<const __half*>(p)[at]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ void store(void* p, int type, int64_t at, float v) {
  if (type == TQ_F32) static_cast<float*>(p)[at] = v;
  else if (type == TQ_F16) static_cast<__half*>(p)[at] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

__global__ void __launch_bounds__(kThreads) lora_kernel(const __grid_constant__ Args p) {
  __shared__ float h[kMaxRank];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const int id = p.ids[t], warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int rank = 0;
  if (id >= 0) {
    const bool known = id < p.l.adapters;
    rank = !known ? -1 : p.l.rank ? p.l.rank[id] : (int)p.l.max_rank;
    if (rank < 0 || rank > p.l.max_rank) {
      if (threadIdx.x == 0) atomicMax(p.status, kDevIndex);
      rank = 0;
    }
  }
  if (rank == 0 && p.z) {   // Z as it is, to the bit
    if (p.z == p.y) return;
    for (int64_t n = threadIdx.x; n < p.l.rows; n += kThreads) {
      const int64_t from = t * p.z_stride + n, to = t * p.y_stride + n;
      if (p.y_type == TQ_F32) static_cast<uint32_t*>(p.y)[to] = static_cast<const uint32_t*>(p.z)[from];
      else static_cast<uint16_t*>(p.y)[to] = static_cast<const uint16_t*>(p.z)[from];
    }
    return;
  }
  const float scale = rank > 0 && p.l.scale ? p.l.scale[id] : 1.0f;
  for (int j = warp; j < rank; j += kThreads / 32) {
    const int64_t row = id * p.l.a_stride + j * p.l.a_row_stride;
    float sum = 0.0f;
    for (int64_t k = lane; k < p.l.cols; k += 32)
      sum = fmaf(load(p.l.a, p.l.type, row + k), load(p.x, p.x_type, t * p.x_stride + k), sum);
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) h[j] = scale * sum;
  }
  __syncthreads();
  for (int64_t n = threadIdx.x; n < p.l.rows; n += kThreads) {
    const int64_t row = id * p.l.b_stride + n * p.l.b_row_stride;
    float sum = 0.0f;
    for (int j = 0; j < rank; ++j) sum = fmaf(load(p.l.b, p.l.type, row + j), h[j], sum);
    if (p.z) sum += load(p.z, p.y_type, t * p.z_stride + n);
    store(p.y, p.y_type, t * p.y_stride + n, sum);
  }
}

}  // namespace

int64_t lora_workspace_bytes(int64_t, int64_t) { return 0; }

cudaError_t launch_lora_add(const LoraCall& c, cudaStream_t s) {
  const Args p = {c.x, c.z, c.y, c.ids, c.lora, c.x_stride, c.z_stride, c.y_stride, c.x_type, c.y_type,
                  c.status};
  return launch_pdl(lora_kernel, dim3((unsigned)c.ntok), dim3(kThreads), 0, s, p);
}

}  // namespace tq
