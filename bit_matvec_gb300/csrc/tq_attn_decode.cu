// tq_attn_decode.cu -- causal attention of a few rows (token, query head) at a
// time over the paged cache: decode, and short drafts.
//
// For a row at position p: s_j = scale q.k_j over the visible keys j <= p,
// o = sum_j 2^(c s_j - M) v_j / sum_j 2^(c s_j - M), c = log2(e), with the
// running maximum M and sum kept in 32 bits (one pass over the keys).
//
// Bound by the bytes of the keys and values: a thread block takes 16 RW rows
// (all query heads that share a key/value head, times a few tokens) and reads
// every key once for all of them. One producer warp streams tiles of K
// and V through a ring of shared-memory stages with TMA boxes, one per page
// piece, 128-byte swizzled so that the fragment loads are free of bank
// conflicts. The four other warps split a tile RW ways by rows (16 rows, one
// matrix fragment, each) and 4 / RW ways by keys, each with its own maximum,
// sum and output accumulators, so that they never wait for one another until
// the merge at the end. mma.sync, not tcgen05: at 16 rows the tensor work is
// 16 flop per byte, far from any rate, and registers give the softmax its
// operands without a trip through TMEM.
// The keys of a row tile are split over thread blocks where there are few of
// them. Up to 8 blocks are a cluster and join their results through one
// another's shared memory; those of more go through the workspace and a second
// kernel, which costs about 3.5 us where the cluster takes 1.
#include "tq_attn_dev.cuh"

namespace tq {
namespace {

constexpr int kWarps = 4;             // compute warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kUp = 15;               // f16 weights are up to 2^kUp

// A stage is 16 KB of keys and 16 KB of values whatever the head's size; three
// of them leave room for two blocks on an SM.
template <int DP> struct Smem {
  static constexpr int kKeys = DP == 128 ? 64 : 128;   // keys of a tile
  static constexpr int kStages = 3;
  static constexpr int kTile = kKeys * DP * 2;         // bytes of a K or V tile
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

// Values at this block's shared address `a` in block s of the cluster.
__device__ __forceinline__ float2 ld_cluster2(uint32_t a, int s) {
  float2 v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %2, %3;\n\t"
      "ld.shared::cluster.v2.f32 {%0, %1}, [r];\n\t}"
      : "=f"(v.x), "=f"(v.y) : "r"(a), "r"(s) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a, int s) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a), "r"(s) : "memory");
  return v;
}
// A release-acquire barrier of all threads of the cluster's blocks.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
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

template <typename T, int DP, int RW>
__global__ void __launch_bounds__(kThreads, 2)
attn_decode_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<DP>;
  constexpr int kRows = 16 * RW;        // rows of the block
  constexpr int KW = kWarps / RW;       // warps along the keys
  constexpr int kKeys = S::kKeys;
  constexpr int kMine = kKeys / KW;     // keys of a tile that a warp takes,
  constexpr int NK = kMine / 16 < 4 ? kMine / 16 : 4;   // in steps of NK x 16
  constexpr int kStages = S::kStages, kSub = DP / 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const basep = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t bars = base + kStages * 2 * S::kTile;   // full[], then empty[]
  volatile int* const failed = reinterpret_cast<volatile int*>(basep + kStages * 2 * S::kTile + 128);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // of a cluster: this block's result, [row][DP] and (maximum, sum) of a row,
  // past the warps' partial results
  constexpr int kPartial = kWarps * 16 * (DP + 6) * 4;
  float* const mine_o = reinterpret_cast<float*>(basep + kPartial);
  float* const mine_l = mine_o + kRows * DP;
  static_assert(kPartial % 16 == 0 && kPartial + kRows * (DP + 2) * 4 <= kStages * 2 * S::kTile, "merge");

  const bool stalled = p.stall_ns > 0 && blockIdx.x == 0 && blockIdx.y == 0;
  const uint64_t limit = stalled ? p.stall_ns : kWaitNs;

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
  const int kv = min(max(p.kv_len[seq], 0), p.max_positions);
  if (threadIdx.x == 0 && tile == 0 && split == 0 && head == 0 &&
      (qn > p.max_q || p.kv_len[seq] > p.max_positions || p.q_start[seq] < 0 ||
       p.q_start[seq] > p.q_start[seq + 1] || p.q_start[seq + 1] > ntok))
    *p.status = kDevIndex;
  const int row0 = tile * kRows;
  const int rows = min(kRows, qn * p.group - row0);
  if (rows <= 0) return;
  // row r of the tile is query head off0 + r of token tok0, running on into the
  // next tokens
  const int tok0 = row0 / p.group, off0 = row0 - tok0 * p.group;
  auto by_group = [&](int x) {
    return p.group_inv ? (int)__umulhi((uint32_t)x, p.group_inv) : x / p.group;
  };
  // positions of the tile's first and last row; keys [lo, hi) are seen by some row
  const int pos_first = kv - qn + tok0, pos_last = pos_first + by_group(off0 + rows - 1);
  const int hi = max(pos_last + 1, 0);
  const int lo = p.window > 0 ? max(0, pos_first - p.window + 1) : 0;
  const int t_lo = lo / kKeys, t_hi = (hi + kKeys - 1) / kKeys;
  const int t0 = min(t_lo + split * p.chunk_tiles, t_hi);
  const int t1 = split == p.nsplit - 1 ? t_hi : min(t0 + p.chunk_tiles, t_hi);

  int issued = 0;   // tiles that the producer requested
  if (warp == kWarps) {
    // ------------------------------------------------ producer
    const int boxes = kKeys / p.box_rows;    // 1 .. 16, one lane each
    const int off = lane * p.box_rows;
    bool bad = false, seen = false;
    int entry = -1, slot = 0;
    // the table's entry for this lane's box of tile t is loaded a tile ahead and
    // looked at when its turn comes; seen: some row sees the box
    auto locate = [&](int t) {
      const int key = t * kKeys + off;
      seen = lane < boxes && t < t1 && key < hi && key + p.box_rows > lo;
      if (seen) {
        const int lp = key / p.page_size;
        slot = key - lp * p.page_size;
        entry = lp < p.table_width ? p.table[seq * p.table_stride + lp] : -1;
      }
    };
    locate(t0);
    int stage = 0, phase = 0;
    for (int t = t0; t < t1 && !stalled; ++t) {
      // the page one past the cache (zeros, nothing read) for a box that no row
      // sees
      int pg = p.pages, sl = 0;
      if (seen) {
        if (entry >= 0 && entry < p.pages) {
          pg = entry;
          sl = slot;
        } else {
          bad = true;
        }
      }
      locate(t + 1);
      // one answer for the warp: lanes whose waits ended apart would part here
      const bool free = t - t0 < kStages ||
                        mbarrier_wait_bounded(bars + 8 * (kStages + stage), phase ^ 1, limit);
      if (!__all_sync(0xffffffffu, free && !*failed)) {
        *failed = 1;
        break;
      }
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
      ++issued;
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (bad) *p.status = kDevIndex;
  } else {
    // ------------------------------------------------ compute warps
    const int g = lane >> 2, tq = lane & 3;
    const int rw = warp / KW, kw = warp % KW;   // the warp's 16 rows and its share of the keys
    const bool busy = rw * 16 < rows;
    // this thread's rows g and g + 8: query fragments and positions
    uint32_t qf[DP / 16][4];
    int pos[2];
    // a negative scale turns the queries and one of zero takes zeros for them,
    // so that the maximum of S is that of the scores and masked ones stay minus
    // infinity
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
    const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);
    const int dim = p.scale_log2 == 0.0f ? 0 : p.dim;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = min(rw * 16 + g + 8 * h, rows - 1);   // rows past the end repeat the last
      const int i = by_group(off0 + r), hh = off0 + r - i * p.group;
      pos[h] = pos_first + i;
      const T* q = static_cast<const T*>(p.q) + (int64_t)(q0 + tok0 + i) * p.q_stride +
                   (int64_t)(head * p.group + hh) * p.dim;
#pragma unroll
      for (int s = 0; s < DP / 16; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = s * 16 + e * 8 + 2 * tq;
          qf[s][h + 2 * e] = d < dim ? *reinterpret_cast<const uint32_t*>(q + d) ^ flip : 0u;
        }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;

    // ldmatrix addresses: matrix mi = lane / 8, row lane % 8 of it
    const int mi = lane >> 3, mr = lane & 7;
    const int krow = kw * kMine + (mi >> 1) * 8 + mr, kchunk = mi & 1;
    const int vrow = kw * kMine + (mi & 1) * 8 + mr, vchunk = mi >> 1;

    int stage = 0, phase = 0;
    bool ok = true;
    for (int t = t0; t < t1; ++t) {
      // (and one answer for the warp, whose matrix instructions want all lanes)
      if (!__all_sync(0xffffffffu, mbarrier_wait_bounded(bars + 8 * stage, phase, limit))) {
        ok = false;
        break;
      }
      const uint32_t ks = base + stage * 2 * S::kTile, vs = ks + S::kTile;
      const int first = t * kKeys + kw * kMine;   // the warp's first key of the tile
      // values of keys that no row sees may be anything: zero them (their
      // weights are zero, but zero times NaN is not)
      if (busy && (first + kMine > hi || first < lo)) {
        for (int i = lane; i < kMine * DP / 8; i += 32) {
          const int r = kw * kMine + i % kMine, c = i / kMine;
          const int key = t * kKeys + r;
          if (key >= hi || key < lo)
            *reinterpret_cast<uint4*>(basep + (vs - base) + (c >> 3) * kKeys * 128 +
                                      swz(r, c & 7)) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
#pragma unroll
      for (int st = 0; st < kMine; st += 16 * NK) {
        const int key0 = first + st;
        if (!busy || key0 >= hi || key0 + 16 * NK <= lo) continue;
        // scores of NK x 16 keys: 2 NK independent accumulators
        float s[2 * NK][4] = {};
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
#pragma unroll
          for (int n = 0; n < NK; ++n) {
            uint32_t b[4];
            ldmatrix4(ks + (d >> 2) * kKeys * 128 + swz(krow + st + n * 16, (d & 3) * 2 + kchunk), b);
            mma16816<T>(s[2 * n], qf[d], b[0], b[1]);
            mma16816<T>(s[2 * n + 1], qf[d], b[2], b[3]);
          }
        // masked ones to minus infinity; maxima, of base-2 logarithms
        float mx[2] = {-INFINITY, -INFINITY};
        const bool masked = key0 + 16 * NK - 1 > pos_first ||
                            (p.window > 0 && key0 <= pos_last - p.window);
        if (masked) {
#pragma unroll
          for (int n = 0; n < 2 * NK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int h = e >> 1, key = key0 + n * 8 + 2 * tq + (e & 1);
              s[n][e] = key > pos[h] || (p.window > 0 && key <= pos[h] - p.window)
                            ? -INFINITY : s[n][e];
              mx[h] = fmaxf(mx[h], s[n][e]);
            }
        } else {
#pragma unroll
          for (int n = 0; n < 2 * NK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
        }
        float corr[2], plus[2];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          const float mn = fmaxf(m[h], mx[h] * scale);
          const float ref = mn == -INFINITY ? 0.0f : mn;
          corr[h] = exp2_approx(m[h] - ref);
          plus[h] = addend<T, kUp>(ref);
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
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          uint32_t a[4];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[e] = exp2_approx(fmaf(s[2 * n + q][e], scale, plus[e >> 1]));
              l[e >> 1] += w[e];
            }
            a[2 * q] = pack2<T>(w[0], w[1]);
            a[2 * q + 1] = pack2<T>(w[2], w[3]);
          }
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) {
            uint32_t b[4];
            ldmatrix4_trans(vs + (d >> 2) * kKeys * 128 + swz(vrow + st + n * 16, (d & 3) * 2 + vchunk), b);
            mma16816<T>(o[2 * d], a, b[0], b[1]);
            mma16816<T>(o[2 * d + 1], a, b[2], b[3]);
          }
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
    for (int h = 0; h < 2; ++h) m[h] -= Scaled<T, kUp>::kUp;
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
      float* const mo = reinterpret_cast<float*>(basep);          // [kw][row][DP + 4]
      constexpr int kLd = DP + 4;
      float* const ml = mo + KW * kRows * kLd;                    // [kw][row][2]
      const int mine = kw * kRows + rw * 16 + g;
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(mo + (mine + 8 * h) * kLd + n * 8 + 2 * tq) =
              make_float2(o[n][2 * h], o[n][2 * h + 1]);
      if (tq == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ml[(mine + 8 * h) * 2] = m[h];
          ml[(mine + 8 * h) * 2 + 1] = l[h];
        }
      }
      named_barrier_sync(1, kWarps * 32);
      // four values of a row a thread
#pragma unroll 2
      for (int i = threadIdx.x; i < rows * (DP / 4); i += kWarps * 32) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        if (d >= p.dim) continue;
        float top = -INFINITY, sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < KW; ++w) top = fmaxf(top, ml[(w * kRows + r) * 2]);
        const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const float f = exp2_approx(ml[(w * kRows + r) * 2] - ref);
          const float4 x = *reinterpret_cast<const float4*>(mo + (w * kRows + r) * kLd + d);
          sum = fmaf(f, ml[(w * kRows + r) * 2 + 1], sum);
          acc.x = fmaf(f, x.x, acc.x);
          acc.y = fmaf(f, x.y, acc.y);
          acc.z = fmaf(f, x.z, acc.z);
          acc.w = fmaf(f, x.w, acc.w);
        }
        if (p.cluster > 1) {
          // this block's result, for the others of the cluster
          *reinterpret_cast<float4*>(mine_o + r * DP + d) = acc;
          if (d == 0) {
            mine_l[2 * r] = top;
            mine_l[2 * r + 1] = sum;
          }
          continue;
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float x[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
        const float lse = sum == 0.0f ? -INFINITY : ref + log2f(sum);
        const int ti = by_group(off0 + r);
        const int64_t tok = q0 + tok0 + ti;
        const int qh = head * p.group + off0 + r - ti * p.group;
        if (p.nsplit > 1) {
          const int64_t at = ((int64_t)split * p.ntok + tok) * p.q_heads + qh;
          *reinterpret_cast<float4*>(p.part_o + at * p.dim + d) = make_float4(x[0], x[1], x[2], x[3]);
          if (d == 0) p.part_lse[at] = lse;
        } else {
          store_out4(p.o, p.o_type, tok * p.o_stride + (int64_t)qh * p.dim + d, x);
          if (d == 0 && p.lse) p.lse[tok * p.q_heads + qh] = lse * kLn2;
        }
      }
    }
  }
  if (p.cluster > 1) {
    __syncwarp();
    cluster_sync();
    // four values of a row a thread, dealt to all blocks of the cluster
    const uint32_t at_o = smem_u32(mine_o), at_l = smem_u32(mine_l);
    if (!*failed && warp < kWarps)
      for (int i = split * kWarps * 32 + threadIdx.x; i < rows * (DP / 4); i += p.cluster * kWarps * 32) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        if (d >= p.dim) continue;
        float2 l[kMaxCluster];
        float4 x[kMaxCluster];
        float top = -INFINITY;
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
          l[s] = make_float2(-INFINITY, 0.0f);
          x[s] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (s < p.cluster) {
            l[s] = ld_cluster2(at_l + 8 * r, s);
            x[s] = ld_cluster4(at_o + 4 * (r * DP + d), s);
          }
          top = fmaxf(top, l[s].x);
        }
        const float ref = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
          const float f = exp2_approx(l[s].x - ref);
          sum = fmaf(f, l[s].y, sum);
          o[0] = fmaf(f, x[s].x, o[0]);
          o[1] = fmaf(f, x[s].y, o[1]);
          o[2] = fmaf(f, x[s].z, o[2]);
          o[3] = fmaf(f, x[s].w, o[3]);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= inv;
        const int ti = by_group(off0 + r);
        const int64_t tok = q0 + tok0 + ti;
        const int qh = head * p.group + off0 + r - ti * p.group;
        store_out4(p.o, p.o_type, tok * p.o_stride + (int64_t)qh * p.dim + d, o);
        if (d == 0 && p.lse)
          p.lse[tok * p.q_heads + qh] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * kLn2;
      }
    __syncwarp();
    cluster_sync();   // no block's shared memory goes before the others have read it
  }
  // after a failed wait the producer's copies are still counted on the full
  // barriers: no block leaves before they have landed
  __syncthreads();
  if (*failed && warp == kWarps && lane < kStages) {
    const int last = last_phase(issued, lane, kStages);
    if (last >= 0) mbarrier_wait_bounded(bars + 8 * lane, last, limit / 10);
  }
}

// ---------------------------------------------------------------- host

template <typename T, int DP, int RW>
cudaError_t launch_decode(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, cudaStream_t s) {
  auto kernel = attn_decode_kernel<T, DP, RW>;
  const cudaError_t e = ensure_dynamic_smem((const void*)kernel, Smem<DP>::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t x = c.kv.nseq * p.tiles_x * p.nsplit;
  if (x > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)x, (unsigned)c.kv.heads);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<DP>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, kmap, vmap);
}

template <typename T, int DP>
cudaError_t launch_decode(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, cudaStream_t s) {
  switch (c.plan.tile_rows) {
    case 16: return launch_decode<T, DP, 1>(p, c, kmap, vmap, s);
    case 32: return launch_decode<T, DP, 2>(p, c, kmap, vmap, s);
    default: return launch_decode<T, DP, 4>(p, c, kmap, vmap, s);
  }
}

template <typename T>
cudaError_t launch_decode(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, cudaStream_t s) {
  return c.kv.head_dim <= 64 ? launch_decode<T, 64>(p, c, kmap, vmap, s)
                             : launch_decode<T, 128>(p, c, kmap, vmap, s);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, cudaStream_t s) {
  return c.kv.type == TQ_F16 ? launch_decode<__half>(p, c, kmap, vmap, s)
                             : launch_decode<__nv_bfloat16>(p, c, kmap, vmap, s);
}

}  // namespace tq
