// tq_attn_chunk.cu -- causal attention of many rows (token, query head) at a
// time over the paged cache, on the tcgen05 tensor cores.
//
// The formulas are those of tq_attn_decode.cu. Bound by the tensor rate: 4 D
// flop for each row and key it sees. A thread block takes 256 rows that share
// a key/value head (all its query heads, consecutive tokens) as two halves of
// 128, and streams 128-key tiles of K and V through a ring of shared-memory
// slots (TMA boxes, one per page piece). For each tile and half:
//   S = Q K^T     tcgen05.mma, both operands in shared memory, S in TMEM;
//   P = 2^(c S - M) one thread per row: no exchange between threads; M moves
//                 only when a row's maximum exceeds it by 2^8 (the quotient at
//                 the end makes any M right), and then O is rescaled in TMEM;
//   O += P V      P as the A operand from TMEM, written over S; V is read
//                 as stored, its 64-value rows being the N-major order.
// While one half's softmax runs, the tensor cores work on the other half.
// Two halves to a block, and not a block each, because K and V then cross
// from L2 once for both: at 128 rows a block they would need about 16 TB/s.
#include <type_traits>

#include "tq_attn_dev.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

using namespace tc;

constexpr int kHalf = 128;            // rows of a half: one warpgroup, one row a thread
constexpr int kRows = 2 * kHalf;
constexpr int kKeys = 128;            // keys of a tile
constexpr int kThreads = 2 * kHalf + 64;   // two softmax warpgroups, an MMA and a TMA warp
constexpr float kGrow = 8.0f;         // a maximum moves when it grew by 2^8

template <int DP> struct Smem {
  static constexpr int kSlots = DP == 128 ? 5 : 8;
  static constexpr int kTile = kKeys * DP * 2;      // bytes of a K or V tile, and of half the queries
  static constexpr int kBars = (2 + kSlots) * kTile;
  static constexpr int kBytes = kBars + 256 + 1024; // + barriers and flags + alignment
};

// K-major operand in 128-byte-swizzled rows of 64 values: 8-row groups 1024
// bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return smem_desc(saddr, 16, 1024) | (2ull << 61);
}
// N-major operand (V: values along N, keys along K): blocks of 64 values a
// tile of kKeys rows apart, groups of 8 keys 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_n(uint32_t saddr) {
  return smem_desc(saddr, kKeys * 128, 1024) | (2ull << 61);
}

// Instruction descriptors: S = Q K^T (both K-major) and O += P V (V N-major,
// bit 16); bf16 is format 1 in bits 7-9 and 10-12.
template <typename T, int DP> struct Desc {
  static constexpr uint32_t kType = std::is_same<T, __nv_bfloat16>::value
                                        ? (1u << 7) | (1u << 10) : 0u;
  static constexpr uint32_t kScores = idesc_f16(kHalf, kKeys) | kType;
  static constexpr uint32_t kOut = idesc_f16(kHalf, DP) | kType | (1u << 16);
};

// 64 columns of this thread's TMEM lane -> registers.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]),
        "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]),
        "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31]), "=f"(r[32]), "=f"(r[33]), "=f"(r[34]),
        "=f"(r[35]), "=f"(r[36]), "=f"(r[37]), "=f"(r[38]), "=f"(r[39]), "=f"(r[40]), "=f"(r[41]),
        "=f"(r[42]), "=f"(r[43]), "=f"(r[44]), "=f"(r[45]), "=f"(r[46]), "=f"(r[47]), "=f"(r[48]),
        "=f"(r[49]), "=f"(r[50]), "=f"(r[51]), "=f"(r[52]), "=f"(r[53]), "=f"(r[54]), "=f"(r[55]),
        "=f"(r[56]), "=f"(r[57]), "=f"(r[58]), "=f"(r[59]), "=f"(r[60]), "=f"(r[61]), "=f"(r[62]),
        "=f"(r[63])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Minus infinity into the scores n of a 64-key piece outside (lo, hi].
__device__ __forceinline__ void mask64(float (&s)[64], int lo, int hi) {
#pragma unroll
  for (int n = 0; n < 64; ++n)
    if (n > hi || n <= lo) s[n] = -INFINITY;
}

__device__ __forceinline__ float max64(const float (&s)[64]) {
  float a = s[0], b = s[1], c = s[2], d = s[3];
#pragma unroll
  for (int n = 4; n < 64; n += 4) {
    a = fmaxf(a, s[n]);
    b = fmaxf(b, s[n + 1]);
    c = fmaxf(c, s[n + 2]);
    d = fmaxf(d, s[n + 3]);
  }
  return fmaxf(fmaxf(a, b), fmaxf(c, d));
}

// Weights of 64 scores, 2^(scale s - ref), packed in pairs of T into TMEM;
// their sum into (l0, l1).
template <typename T>
__device__ __forceinline__ void weights64(const float (&s)[64], uint64_t scale2, uint64_t ref2,
                                          uint64_t& l0, uint64_t& l1, uint32_t taddr) {
  uint32_t w[32];
#pragma unroll
  for (int n = 0; n < 32; ++n) {
    const float2 x = f2_unpack(f2_fma(f2_packf(s[2 * n], s[2 * n + 1]), scale2, ref2));
    const float a = exp2_approx(x.x), b = exp2_approx(x.y);
    if (n & 1) l1 = f2_add(l1, f2_packf(a, b));
    else l0 = f2_add(l0, f2_packf(a, b));
    w[n] = pack2<T>(a, b);
  }
  tmem_st32(taddr, w);
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_chunk_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<DP>;
  constexpr int kSlots = S::kSlots, kSub = DP / 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const basep = smem_raw + (base - smem_u32(smem_raw));
  // queries of the two halves, then the ring, then the barriers
  const uint32_t ring = base + 2 * S::kTile;
  const uint32_t bars = base + S::kBars;
  const uint32_t full = bars, empty = bars + 8 * kSlots, q_full = empty + 8 * kSlots;
  const uint32_t s_full = q_full + 8, p_ready = s_full + 16, drain = p_ready + 16;
  volatile uint32_t* const shared = reinterpret_cast<volatile uint32_t*>(basep + S::kBars + 192);
  volatile uint32_t* const failed = shared + 1;   // shared[0]: TMEM address, [2]: sequence
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbarrier_init(full + 8 * i, 1);
      mbarrier_init(empty + 8 * i, 1);
    }
    mbarrier_init(q_full, 2 * kHalf);
    for (int i = 0; i < 2; ++i) {
      mbarrier_init(s_full + 8 * i, 1);
      mbarrier_init(p_ready + 8 * i, 4);
    }
    mbarrier_init(drain, 1);
    *failed = 0;
    mbarrier_init_fence();
  }
  if (warp == 8) {
    tmem_alloc<1>(smem_u32(const_cast<uint32_t*>(shared)), 512);
    tmem_relinquish<1>();
  }
  pdl_wait_primary();
  pdl_launch_dependents();

  // The block's row tile. The tiles of sequence b are numbered from
  // f(b) = floor(q_start[b] * group / kRows) + b, which leaves each sequence
  // room for all of its own; the last (longest) tiles start first.
  const int head = blockIdx.y;
  const int split = blockIdx.x % p.nsplit;
  const int64_t slot = p.tiles_x - 1 - (int64_t)(blockIdx.x / p.nsplit);
  const int ntok = (int)p.ntok;
  auto first_slot = [&](int b) {
    const int64_t q = min(max(p.q_start[b], 0), ntok);
    return q * p.group / kRows + b;
  };
  if (warp == 9) {
    int lo = 0, hi = p.nseq;   // f(lo) <= slot < f(hi): 32 probes a step
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + lane * step;
      const uint32_t below = __ballot_sync(0xffffffffu, at < hi && first_slot(at) <= slot);
      const int n = max(__popc(below), 1);
      lo += (n - 1) * step;
      hi = min(lo + step, hi);
    }
    if (lane == 0) shared[2] = (uint32_t)lo;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = shared[0];
  const int seq = (int)shared[2];
  const int q0 = min(max(p.q_start[seq], 0), ntok);
  const int qn = min(max(p.q_start[seq + 1], q0), ntok) - q0;
  const int kv = max(p.kv_len[seq], 0);
  const int64_t tile = slot - first_slot(seq);
  const int64_t row0 = tile * kRows;
  const int rows = (int)min((int64_t)kRows, (int64_t)qn * p.group - row0);
  if (tile == 0 && split == 0 && head == 0 && threadIdx.x == 0 &&
      (qn > p.max_q || (int64_t)kv > p.table_width * p.page_size))
    *p.status = kDevIndex;
  const int tok0 = rows > 0 ? (int)(row0 / p.group) : 0;      // the tile's first token
  const int off0 = rows > 0 ? (int)(row0 - (int64_t)tok0 * p.group) : 0;
  // keys [lo, hi) are seen by some row
  const int pos_first = kv - qn + tok0;
  const int pos_last = rows > 0 ? kv - qn + tok0 + (off0 + rows - 1) / p.group : -1;
  const int hi = max(pos_last + 1, 0);
  const int lo = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos_first - p.window + 1) : 0;
  const int t_lo = lo / kKeys, t_hi = (hi + kKeys - 1) / kKeys;
  const int t0 = min(t_lo + split * p.chunk_tiles, t_hi);
  const int t1 = rows <= 0 ? t0 : split == p.nsplit - 1 ? t_hi : min(t0 + p.chunk_tiles, t_hi);
  const int nt = t1 - t0;
  const bool two = rows > kHalf;

  if (nt > 0) {
    if (warp == 9) {
      // ------------------------------------------------ TMA producer
      const int boxes = kKeys / p.box_rows;   // 1 .. 16, one lane each
      const int off = lane * p.box_rows;
      bool bad = false;
      int page = p.pages, pslot = 0;
      // page and slot of this lane's box of tile t; the page one past the
      // cache (zeros, nothing read) where no row sees the box
      auto locate = [&](int t) {
        const int key = t * kKeys + off;
        page = p.pages;
        pslot = 0;
        if (lane < boxes && t < t1 && key < hi && key + p.box_rows > lo) {
          const int lp = key / p.page_size;
          pslot = key - lp * p.page_size;
          int pg = -1;
          if (lp < p.table_width) pg = p.table[seq * p.table_stride + lp];
          if (pg >= 0 && pg < p.pages) page = pg;
          else bad = true;
        }
      };
      locate(t0);
      int it = 0;
      for (int j = 0; j < nt && !*failed; ++j) {
        const int pg = page, sl = pslot;
        locate(t0 + j + 1);
        for (int v = 0; v < 2; ++v, ++it) {
          const int sidx = it % kSlots;
          if (it >= kSlots && !mbarrier_wait_bounded(empty + 8 * sidx, (it / kSlots - 1) & 1, kWaitNs)) {
            *failed = 1;
            break;
          }
          if (lane == 0) mbarrier_arrive_expect_tx(full + 8 * sidx, S::kTile);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = ring + sidx * S::kTile + off * 128;
#pragma unroll
            for (int c = 0; c < kSub; ++c)
              tma_box(dst + c * kKeys * 128, v ? &vmap : &kmap, c * 64, sl, head, pg, full + 8 * sidx);
          }
        }
      }
      if (bad) *p.status = kDevIndex;
      __syncwarp();
      // no block leaves before its copies have landed
      if (*failed && lane < kSlots && it > lane)
        mbarrier_wait_bounded(full + 8 * lane, ((it - 1 - lane) / kSlots) & 1, kWaitNs / 10);
    } else if (warp == 8) {
      // ------------------------------------------------ MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc_s = Desc<T, DP>::kScores, idesc_o = Desc<T, DP>::kOut;
        auto qk = [&](int h, int item) {
          const uint32_t a = base + h * S::kTile, b = ring + (item % kSlots) * S::kTile;
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) {
            const uint32_t o = (d >> 2) * kKeys * 128 + (d & 3) * 32;
            mma_f16_ss(tmem + h * kKeys, desc_k(a + o), desc_k(b + o), idesc_s, d > 0);
          }
        };
        auto pv = [&](int h, int item, bool first) {
          const uint32_t b = ring + (item % kSlots) * S::kTile;
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_f16_tmem_a(tmem + 256 + h * DP, tmem + h * kKeys + k * 8, desc_n(b + k * 2048), idesc_o,
                           !(first && k == 0));
        };
        auto wait = [&](uint32_t bar, uint32_t parity) {
          if (*failed || !mbarrier_wait_bounded(bar, parity, kWaitNs)) {
            *failed = 1;
            return false;
          }
          return true;
        };
        auto wait_item = [&](int item) { return wait(full + 8 * (item % kSlots), (item / kSlots) & 1); };
        bool ok = wait(q_full, 0) && wait_item(0);
        if (ok) {
          tc_fence_after();
          qk(0, 0);
          mma_commit(s_full);
          if (two) {
            qk(1, 0);
            mma_commit(s_full + 8);
          }
          mma_commit(empty);
        }
        for (int j = 0; j < nt && ok; ++j) {
          const int vi = 2 * j + 1, ki = 2 * j + 2;
          const bool more = j + 1 < nt;
          ok = wait_item(vi) && wait(p_ready, j & 1);
          if (!ok) break;
          tc_fence_after();
          pv(0, vi, j == 0);
          if (more) {
            ok = wait_item(ki);
            if (!ok) break;
            qk(0, ki);
          }
          mma_commit(s_full);
          if (two) {
            ok = wait(p_ready + 8, j & 1);
            if (!ok) break;
            tc_fence_after();
            pv(1, vi, j == 0);
            mma_commit(empty + 8 * (vi % kSlots));
            if (more) qk(1, ki);
            mma_commit(s_full + 8);
          } else {
            mma_commit(empty + 8 * (vi % kSlots));
          }
          if (more) mma_commit(empty + 8 * (ki % kSlots));
        }
        if (*failed) {   // the MMAs issued end before TMEM is freed
          mma_commit(drain);
          mbarrier_wait_bounded(drain, 0, kWaitNs / 10);
        }
      }
      __syncwarp();
    }
  }

  if (warp < 8) {
    // -------------------------------------------------- softmax, one row a thread
    const int h = warp >> 2;                          // half
    const int r = threadIdx.x;                        // row of the tile
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lane_base + h * kKeys, to = lane_base + 256 + h * DP;
    // a negative scale turns the queries, so that the maximum is one of S; a
    // zero one takes zero queries
    const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);
    if (nt > 0) {
      const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      for (int i = threadIdx.x; i < kRows * (DP / 8); i += 2 * kHalf) {
        const int row = i / (DP / 8), c = i % (DP / 8);
        uint4 x = zero;
        if (row < rows && c * 8 < p.dim && p.scale_log2 != 0.0f) {
          const int t = (off0 + row) / p.group, hh = (off0 + row) - t * p.group;
          const T* q = static_cast<const T*>(p.q) + (int64_t)(q0 + tok0 + t) * p.q_stride +
                       (int64_t)(head * p.group + hh) * p.dim + c * 8;
          x = *reinterpret_cast<const uint4*>(q);
          x.x ^= flip;
          x.y ^= flip;
          x.z ^= flip;
          x.w ^= flip;
        }
        *reinterpret_cast<uint4*>(basep + (row / kHalf) * S::kTile + (c >> 3) * kHalf * 128 +
                                  swz(row % kHalf, c & 7)) = x;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbarrier_arrive(q_full);
    }
    const int trow = (off0 + min(r, max(rows, 1) - 1)) / p.group;
    const int pos = kv - qn + tok0 + trow;
    float m = -INFINITY;
    uint64_t l0 = 0, l1 = 0;
    const uint64_t scale2 = f2_packf(scale, scale);
    bool ok = true;
    if (h == 0 || two) {
      for (int j = 0; j < nt; ++j) {
        if (*failed || !mbarrier_wait_bounded(s_full + 8 * h, j & 1, kWaitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int key0 = (t0 + j) * kKeys;
        float a[64], b[64];
        tmem_ld64(ts, a);
        tmem_ld64(ts + 64, b);
        // the row sees the keys (pos - window, pos]
        const int see = pos - key0;
        const int64_t from = p.window > 0 ? (int64_t)pos - p.window - key0 : -1;
        if (__any_sync(0xffffffffu, see < kKeys - 1 || from >= 0)) {
          const int f = (int)max(from, (int64_t)-1);
          mask64(a, f, see);
          mask64(b, f - 64, see - 64);
        }
        const float top = fmaxf(max64(a), max64(b)) * scale;
        if (__any_sync(0xffffffffu, top > m + kGrow || (m == -INFINITY && top > m))) {
          const float mn = fmaxf(m, top);
          const float corr = exp2_approx(m - (mn == -INFINITY ? 0.0f : mn));
          m = mn;
          const uint64_t c2 = f2_packf(corr, corr);
          l0 = f2_mul(l0, c2);
          l1 = f2_mul(l1, c2);
          if (j > 0) {
#pragma unroll
            for (int c = 0; c < DP; c += 32) {
              uint32_t o[32];
              tmem_ld32(to + c, o);
#pragma unroll
              for (int n = 0; n < 32; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * corr);
              tmem_st32(to + c, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.0f : -m;
        const uint64_t ref2 = f2_packf(ref, ref);
        weights64<T>(a, scale2, ref2, l0, l1, ts);
        weights64<T>(b, scale2, ref2, l0, l1, ts + 32);
        // values of keys that no row sees may be anything: zero them (their
        // weights are zero, but zero times NaN is not)
        if (h == 0 && (key0 + kKeys > hi || key0 < lo)) {
          const int item = 2 * j + 1;
          if (!mbarrier_wait_bounded(full + 8 * (item % kSlots), (item / kSlots) & 1, kWaitNs)) {
            ok = false;
            break;
          }
          const int key = key0 + r;
          if (key >= hi || key < lo) {
            uint8_t* v = basep + (2 + item % kSlots) * S::kTile;
#pragma unroll
            for (int c = 0; c < DP / 8; ++c)
              *reinterpret_cast<uint4*>(v + (c >> 3) * kKeys * 128 + swz(r, c & 7)) =
                  make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbarrier_arrive(p_ready + 8 * h);
      }
      if (ok && nt > 0 && !mbarrier_wait_bounded(s_full + 8 * h, nt & 1, kWaitNs)) ok = false;
      if (!ok) *failed = 1;
      tc_fence_after();
      __syncwarp();
      if (ok && !*failed) {
        // ---------------------------------------------- output rows
        const float2 la = f2_unpack(f2_add(l0, l1));
        const float l = la.x + la.y;
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        const float lse = l > 0.0f ? m + log2f(l) : -INFINITY;
        const bool live = r < rows;
        const int64_t tok = q0 + tok0 + trow;
        const int qh = head * p.group + (off0 + r) % p.group;
        const int64_t at = p.nsplit > 1 ? ((int64_t)split * p.ntok + tok) * p.q_heads + qh : 0;
        if (live && p.nsplit > 1) p.part_lse[at] = lse;
        if (live && p.nsplit == 1 && p.lse) p.lse[tok * p.q_heads + qh] = lse * kLn2;
        const int64_t obase = tok * p.o_stride + (int64_t)qh * p.dim;
#pragma unroll
        for (int c = 0; c < DP; c += 32) {
          uint32_t o[32] = {};
          if (nt > 0) tmem_ld32(to + c, o);
          if (!live) continue;
#pragma unroll
          for (int n = 0; n < 32; n += 4) {
            if (c + n >= p.dim) continue;
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = nt > 0 ? __uint_as_float(o[n + e]) * inv : 0.0f;
            if (p.nsplit > 1)
              *reinterpret_cast<float4*>(p.part_o + at * p.dim + c + n) =
                  make_float4(x[0], x[1], x[2], x[3]);
            else
              store_out4(p.o, p.o_type, obase + c + n, x);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*failed && threadIdx.x == 0) *p.status = kDevTimeout;
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 512);
  }
}

template <typename T, int DP>
cudaError_t launch_chunk(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, cudaStream_t s) {
  auto kernel = attn_chunk_kernel<T, DP>;
  const cudaError_t e = ensure_dynamic_smem((const void*)kernel, Smem<DP>::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t x = c.plan.tiles_x * p.nsplit;
  if (x > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(kernel, dim3((unsigned)x, (unsigned)c.kv.heads), dim3(kThreads),
                    Smem<DP>::kBytes, s, p, kmap, vmap);
}

template <typename T>
cudaError_t launch_chunk(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, cudaStream_t s) {
  return c.kv.head_dim <= 64 ? launch_chunk<T, 64>(p, c, kmap, vmap, s)
                             : launch_chunk<T, 128>(p, c, kmap, vmap, s);
}

}  // namespace

cudaError_t launch_attn_chunk(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                              const CUtensorMap& vmap, cudaStream_t s) {
  return c.kv.type == TQ_F16 ? launch_chunk<__half>(p, c, kmap, vmap, s)
                             : launch_chunk<__nv_bfloat16>(p, c, kmap, vmap, s);
}

}  // namespace tq
