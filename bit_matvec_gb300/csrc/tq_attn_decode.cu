// tq_attn_decode.cu -- causal attention of a few rows (token, query head) at a
// time over the paged cache: decode, and short drafts.
//
// For a row at position p: s_j = scale q.k_j over the visible keys j <= p,
// o = sum_j 2^(c s_j - M) v_j / sum_j 2^(c s_j - M), c = log2(e), with the
// running maximum M and sum kept in 32 bits (one pass over the keys).
//
// Bound by the bytes of the keys and values: a thread block takes the 16 rows
// of a 16-row matrix fragment (all query heads that share a key/value head,
// times a few tokens) and reads every key once for all of them. One producer
// warp streams 64-key tiles of K and V through a ring of shared-memory stages
// with TMA boxes, one per page piece, 128-byte swizzled so that the fragment
// loads are free of bank conflicts. Each of the four other warps owns 16 of a
// tile's 64 keys with its own maximum, sum and output accumulators, so the
// warps never wait for one another until the merge at the end. mma.sync, not
// tcgen05: at 16 rows the tensor work is 16 flop per byte, far from any rate,
// and registers give the softmax its operands without a trip through TMEM.
// The keys of a row tile are split over thread blocks where there are few of
// them; partial results are joined by a second kernel.
#include <cuda.h>

#include "tq_attn.cuh"

namespace tq {
namespace {

constexpr int kRows = 16;
constexpr int kKeys = 64;             // keys of a stage
constexpr int kWarps = 4;             // compute warps, 16 keys of a stage each
constexpr int kThreads = (kWarps + 1) * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitNs = 1000000000ull;

struct Params {
  const void* q;
  void* o;
  float* lse;
  float* part_o;
  float* part_lse;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t q_stride, o_stride, table_stride, table_width;
  int64_t ntok;
  int* status;
  int q_heads, group, dim, page_size, pages, box_rows;
  int nseq, tiles_x, nsplit, chunk_tiles, max_q;
  int o_type;
  int64_t window;
  float scale_log2;
};

template <int DP> struct Smem {
  static constexpr int kStages = DP == 128 ? 3 : 6;
  static constexpr int kTile = kKeys * DP * 2;      // bytes of a K or V tile
  static constexpr int kBytes = kStages * 2 * kTile + 1024 + 256;   // + alignment + barriers
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4],
                                                 uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 2)
attn_decode_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<DP>;
  constexpr int kStages = S::kStages, kSub = DP / 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const basep = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t bars = base + kStages * 2 * S::kTile;   // full[], then empty[]
  volatile int* const failed = reinterpret_cast<volatile int*>(basep + kStages * 2 * S::kTile + 128);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbarrier_init(bars + 8 * i, 1);
      mbarrier_init(bars + 8 * (kStages + i), kWarps);
    }
    *failed = 0;
    mbarrier_init_fence();
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  __syncthreads();

  // the block's row tile and key range
  const int head = blockIdx.y;
  const int split = blockIdx.x % p.nsplit;
  const int rest = blockIdx.x / p.nsplit;
  const int tile = rest % p.tiles_x, seq = rest / p.tiles_x;
  const int ntok = (int)p.ntok;
  const int q0 = min(max(p.q_start[seq], 0), ntok);
  const int qn = min(max(p.q_start[seq + 1], q0), ntok) - q0;
  const int kv = max(p.kv_len[seq], 0);
  if (threadIdx.x == 0 && tile == 0 && split == 0 && head == 0 &&
      (qn > p.max_q || (int64_t)kv > p.table_width * p.page_size))
    *p.status = kDevIndex;
  const int row0 = tile * kRows;
  const int rows = min(kRows, qn * p.group - row0);
  if (rows <= 0) return;
  // positions of the tile's first and last row; keys [lo, hi) are seen by some row
  const int pos_first = kv - qn + row0 / p.group, pos_last = kv - qn + (row0 + rows - 1) / p.group;
  const int hi = max(pos_last + 1, 0);
  const int lo = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos_first - p.window + 1) : 0;
  const int t_lo = lo / kKeys, t_hi = (hi + kKeys - 1) / kKeys;
  const int t0 = min(t_lo + split * p.chunk_tiles, t_hi);
  const int t1 = split == p.nsplit - 1 ? t_hi : min(t0 + p.chunk_tiles, t_hi);

  if (warp == kWarps) {
    // ------------------------------------------------ producer
    const int boxes = kKeys / p.box_rows;    // 1 .. 8, one lane each
    const int off = lane * p.box_rows;
    int page = p.pages, slot = 0;
    bool bad = false;
    // page and slot of this lane's box of tile t; the page one past the cache
    // (zeros, nothing read) where no row sees the box
    auto locate = [&](int t) {
      const int key = t * kKeys + off;
      page = p.pages;
      slot = 0;
      if (lane < boxes && t < t1 && key < hi && key + p.box_rows > lo) {
        const int lp = key / p.page_size;
        slot = key - lp * p.page_size;
        int pg = -1;
        if (lp < p.table_width) pg = p.table[seq * p.table_stride + lp];
        if (pg >= 0 && pg < p.pages) page = pg;
        else bad = true;
      }
    };
    locate(t0);
    int stage = 0, phase = 0;
    for (int t = t0; t < t1; ++t) {
      const int pg = page, sl = slot;
      locate(t + 1);
      if (t - t0 >= kStages &&
          !mbarrier_wait_bounded(bars + 8 * (kStages + stage), phase ^ 1, kWaitNs)) {
        *failed = 1;
        break;
      }
      if (*failed) break;
      const uint32_t full = bars + 8 * stage;
      if (lane == 0) mbarrier_arrive_expect_tx(full, 2 * S::kTile);
      __syncwarp();
      if (lane < boxes) {
        const uint32_t k = base + stage * 2 * S::kTile + off * 128, v = k + S::kTile;
#pragma unroll
        for (int c = 0; c < kSub; ++c) {
          tma_box(k + c * kKeys * 128, &kmap, c * 64, sl, head, pg, full);
          tma_box(v + c * kKeys * 128, &vmap, c * 64, sl, head, pg, full);
        }
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (bad) *p.status = kDevIndex;
  } else {
    // ------------------------------------------------ compute warps
    const int g = lane >> 2, tq = lane & 3;
    // this thread's rows g and g + 8: query fragments and positions
    uint32_t qf[DP / 16][4];
    int pos[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = min(g + 8 * h, rows - 1);   // rows past the end repeat the last
      const int i = (row0 + r) / p.group, hh = (row0 + r) % p.group;
      pos[h] = kv - qn + i;
      const T* q = static_cast<const T*>(p.q) + (int64_t)(q0 + i) * p.q_stride +
                   (int64_t)(head * p.group + hh) * p.dim;
#pragma unroll
      for (int s = 0; s < DP / 16; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = s * 16 + e * 8 + 2 * tq;
          qf[s][h + 2 * e] = d < p.dim ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
        }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;

    // ldmatrix addresses: matrix mi = lane / 8, row lane % 8 of it
    const int mi = lane >> 3, mr = lane & 7;
    const int krow = warp * 16 + (mi >> 1) * 8 + mr, kchunk = mi & 1;
    const int vrow = warp * 16 + (mi & 1) * 8 + mr, vchunk = mi >> 1;

    int stage = 0, phase = 0;
    bool ok = true;
    for (int t = t0; t < t1; ++t) {
      if (!mbarrier_wait_bounded(bars + 8 * stage, phase, kWaitNs)) {
        ok = false;
        break;
      }
      const uint32_t ks = base + stage * 2 * S::kTile, vs = ks + S::kTile;
      const int key0 = t * kKeys + warp * 16;
      if (key0 < hi && key0 + 16 > lo) {
        float s[2][4] = {};
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          uint32_t b[4];
          ldmatrix4(ks + (d >> 2) * kKeys * 128 + swz(krow, (d & 3) * 2 + kchunk), b);
          mma16816<T>(s[0], qf[d], b[0], b[1]);
          mma16816<T>(s[1], qf[d], b[2], b[3]);
        }
        // values of keys that no row sees may be anything: zero them (their
        // weights are zero, but zero times NaN is not)
        if (key0 + 16 > hi || key0 < lo) {
          for (int i = lane; i < 16 * DP / 8; i += 32) {
            const int r = warp * 16 + i % 16, c = i / 16;
            const int key = t * kKeys + r;
            if (key >= hi || key < lo)
              *reinterpret_cast<uint4*>(basep + (vs - base) + (c >> 3) * kKeys * 128 +
                                        swz(r, c & 7)) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        // scores in base-2 logarithms; masked ones to minus infinity
        float mx[2] = {-INFINITY, -INFINITY};
        const bool masked = key0 + 15 > pos_first ||
                            (p.window > 0 && (int64_t)key0 <= (int64_t)pos_last - p.window);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = e >> 1, key = key0 + n * 8 + 2 * tq + (e & 1);
            float x = s[n][e] * p.scale_log2;
            if (masked && (key > pos[h] ||
                           (p.window > 0 && (int64_t)key <= (int64_t)pos[h] - p.window)))
              x = -INFINITY;
            s[n][e] = x;
            mx[h] = fmaxf(mx[h], x);
          }
        float corr[2], ref[2];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          const float mn = fmaxf(m[h], mx[h]);
          ref[h] = mn == -INFINITY ? 0.0f : mn;
          corr[h] = exp2_approx(m[h] - ref[h]);
          grow |= mn > m[h];
          m[h] = mn;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            o[n][0] *= corr[0];
            o[n][1] *= corr[0];
            o[n][2] *= corr[1];
            o[n][3] *= corr[1];
          }
          l[0] *= corr[0];
          l[1] *= corr[1];
        }
        uint32_t a[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = exp2_approx(s[n][e] - ref[e >> 1]);
            l[e >> 1] += w[e];
          }
          a[2 * n] = pack2<T>(w[0], w[1]);
          a[2 * n + 1] = pack2<T>(w[2], w[3]);
        }
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          uint32_t b[4];
          ldmatrix4_trans(vs + (d >> 2) * kKeys * 128 + swz(vrow, (d & 3) * 2 + vchunk), b);
          mma16816<T>(o[2 * d], a, b[0], b[1]);
          mma16816<T>(o[2 * d + 1], a, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbarrier_arrive(bars + 8 * (kStages + stage));
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) *failed = 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    // ------------------------------------------------ merge of the warps
    // every copy has landed and every warp is done with the stages
    named_barrier_sync(1, kWarps * 32);
    if (*failed) {
      if (threadIdx.x == 0) *p.status = kDevTimeout;
    } else {
      float* const mo = reinterpret_cast<float*>(basep);          // [warp][row][DP + 4]
      constexpr int kLd = DP + 4;
      float* const ml = mo + kWarps * kRows * kLd;                // [warp][row][2]
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(mo + (warp * kRows + g + 8 * h) * kLd + n * 8 + 2 * tq) =
              make_float2(o[n][2 * h], o[n][2 * h + 1]);
      if (tq == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ml[(warp * kRows + g + 8 * h) * 2] = m[h];
          ml[(warp * kRows + g + 8 * h) * 2 + 1] = l[h];
        }
      }
      named_barrier_sync(1, kWarps * 32);
      for (int i = threadIdx.x; i < rows * DP; i += kWarps * 32) {
        const int r = i / DP, d = i % DP;
        if (d >= p.dim) continue;
        float top = -INFINITY, sum = 0.0f, acc = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[(w * kRows + r) * 2]);
        const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = exp2_approx(ml[(w * kRows + r) * 2] - ref);
          sum += f * ml[(w * kRows + r) * 2 + 1];
          acc += f * mo[(w * kRows + r) * kLd + d];
        }
        const float val = sum > 0.0f ? acc / sum : 0.0f;
        const float lse = sum > 0.0f ? ref + log2f(sum) : -INFINITY;
        const int64_t tok = q0 + (row0 + r) / p.group;
        const int qh = head * p.group + (row0 + r) % p.group;
        if (p.nsplit > 1) {
          const int64_t at = ((int64_t)split * p.ntok + tok) * p.q_heads + qh;
          p.part_o[at * p.dim + d] = val;
          if (d == 0) p.part_lse[at] = lse;
        } else {
          store_out(p.o, p.o_type, tok * p.o_stride + (int64_t)qh * p.dim + d, val);
          if (d == 0 && p.lse) p.lse[tok * p.q_heads + qh] = lse * 0.6931471805599453f;
        }
      }
    }
  }
  // after a failed wait the producer's copies are still counted on the full
  // barriers: no block leaves before they have landed
  __syncthreads();
  if (*failed && threadIdx.x < kStages) {
    const int issued = (t1 - t0 - (int)threadIdx.x + kStages - 1) / kStages;
    if (issued > 0) mbarrier_wait_bounded(bars + 8 * threadIdx.x, (issued - 1) & 1, kWaitNs / 10);
  }
}

// Joins the partial results of the splits: o = sum_s 2^(lse_s - M) o_s /
// sum_s 2^(lse_s - M), one warp per row of one query head. Reads
// nsplit * (dim + 1) * 4 bytes a row, a few percent of the keys' bytes.
__global__ void __launch_bounds__(128)
attn_join_kernel(const __grid_constant__ Params p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t rows = p.ntok * p.q_heads;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int64_t tok = row / p.q_heads;
  // tokens past the last sequence's are not written
  if (tok >= p.q_start[p.nseq]) return;
  float top = -INFINITY;
  for (int s = lane; s < p.nsplit; s += 32) top = fmaxf(top, p.part_lse[s * rows + row]);
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float sum = 0.0f, acc[kMaxKvDim / 32] = {};
  if (top != -INFINITY)
    for (int s = 0; s < p.nsplit; ++s) {
      const float f = exp2_approx(p.part_lse[s * rows + row] - top);
      if (f == 0.0f) continue;
      sum += f;
#pragma unroll
      for (int i = 0; i < kMaxKvDim / 32; ++i)
        if (lane + 32 * i < p.dim)
          acc[i] += f * p.part_o[(s * rows + row) * p.dim + lane + 32 * i];
    }
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxKvDim / 32; ++i)
    if (lane + 32 * i < p.dim)
      store_out(p.o, p.o_type, tok * p.o_stride + (row - tok * p.q_heads) * p.dim + lane + 32 * i,
                acc[i] * inv);
  if (lane == 0 && p.lse)
    p.lse[row] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// ---------------------------------------------------------------- host

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn* out) {
  static EncodeFn fn = nullptr;   // the driver's entry point: the same for every call
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeFn>(f);
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
  const CUresult r =
      fn(map, c.type == TQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
         4, p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int DP>
cudaError_t launch_decode(const Params& p, const AttnCall& c, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, cudaStream_t s) {
  auto kernel = attn_decode_kernel<T, DP>;
  const cudaError_t e = ensure_dynamic_smem((const void*)kernel, Smem<DP>::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t x = c.kv.nseq * p.tiles_x * p.nsplit;
  if (x > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(kernel, dim3((unsigned)x, (unsigned)c.kv.heads), dim3(kThreads),
                    Smem<DP>::kBytes, s, p, kmap, vmap);
}

template <typename T>
cudaError_t launch_decode(const Params& p, const AttnCall& c, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, cudaStream_t s) {
  return c.kv.head_dim <= 64 ? launch_decode<T, 64>(p, c, kmap, vmap, s)
                             : launch_decode<T, 128>(p, c, kmap, vmap, s);
}

}  // namespace

cudaError_t launch_attention(const AttnCall& c, cudaStream_t s) {
  Params p = {};
  p.q = c.q;
  p.o = c.o;
  p.lse = c.lse;
  p.part_o = c.part_o;
  p.part_lse = c.part_lse;
  p.q_start = c.q_start;
  p.kv_len = c.kv_len;
  p.table = c.kv.block_table;
  p.q_stride = c.q_stride;
  p.o_stride = c.o_stride;
  p.table_stride = c.kv.table_stride;
  p.table_width = c.kv.table_width;
  p.ntok = c.ntok;
  p.status = c.status;
  p.q_heads = (int)c.q_heads;
  p.group = (int)(c.q_heads / c.kv.heads);
  p.dim = (int)c.kv.head_dim;
  p.page_size = (int)c.kv.page_size;
  p.pages = (int)c.kv.pages;
  // boxes are pieces of a page and of a 64-key tile
  p.box_rows = (int)(c.kv.page_size & -c.kv.page_size);
  if (p.box_rows > kKeys) p.box_rows = kKeys;
  p.nseq = (int)c.kv.nseq;
  p.tiles_x = (int)c.plan.tiles_x;
  p.nsplit = c.plan.nsplit;
  p.chunk_tiles = c.plan.chunk_tiles;
  p.max_q = (int)c.max_q;
  p.o_type = c.o_type;
  p.window = c.window;
  p.scale_log2 = c.scale * kLog2e;
  CUtensorMap kmap, vmap;
  cudaError_t e = cache_map(&kmap, c.kv, c.kv.k, p.box_rows);
  if (e == cudaSuccess) e = cache_map(&vmap, c.kv, c.kv.v, p.box_rows);
  if (e != cudaSuccess) return e;
  e = c.kv.type == TQ_F16 ? launch_decode<__half>(p, c, kmap, vmap, s)
                          : launch_decode<__nv_bfloat16>(p, c, kmap, vmap, s);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  const int64_t grid = (c.ntok * c.q_heads + 3) / 4;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(attn_join_kernel, dim3((unsigned)grid), dim3(128), 0, s, p);
}

}  // namespace tq
