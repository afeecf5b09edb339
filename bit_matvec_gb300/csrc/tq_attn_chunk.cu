// tq_attn_chunk.cu -- causal attention of many rows (token, query head) at a
// time over the paged cache, on the tcgen05 tensor cores.
//
// The formulas are those of tq_attn_decode.cu. Bound by the tensor rate: 4 D
// flop for each row and key it sees. A row tile is up to 256 rows that share a
// key/value head (all its query heads, consecutive tokens). A thread block
// streams 128-key tiles of K and V through a ring of shared-memory slots (TMA
// boxes, one per page piece) and keeps two softmaxes of 128 rows going:
//   S = Q K^T     tcgen05.mma, both operands in shared memory, S in TMEM;
//   P = 2^(c S - M) one thread a row: no exchange between threads (two a row
//                 measured 1.4 times slower: the fixed work of a step
//                 doubles); M moves only when a row's maximum exceeds it by
//                 2^8 (the quotient at the end makes any M right), and then O
//                 is rescaled in TMEM;
//   O += P V      P as the A operand from TMEM, written over S; V is read
//                 as stored, its 64-value rows being the N-major order.
// While one softmax runs, the tensor cores work for the other. With more than
// 128 rows the two are the halves of the row tile, on the same keys: K and V
// then cross from L2 once for both (at 128 rows a block they would need about
// 16 TB/s). With up to 128 rows both take the same rows, on alternate key
// tiles, and are merged at the end.
//
// Blocks find their piece of the work from q_start and kv_len on the device
// (tq_attn_work.cuh). Cut row tiles leave partial results, which a second
// kernel joins.
#include <type_traits>

#include "tq_attn_dev.cuh"
#include "tq_attn_work.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

using namespace tc;
using namespace work;

constexpr int kSoft = 256;            // softmax threads, one a row
constexpr int kThreads = kSoft + 128; // and an MMA, a TMA and a scheduling warp (and one that idles)
constexpr float kGrow = 8.0f;         // a maximum moves when it grew by 2^8
constexpr int kUp = 7;                // f16 weights are up to 2^(kGrow + kUp)
constexpr int kQueue = 4;             // segments the scheduling warp may be ahead
constexpr int kCachedSeqs = 48;       // lengths of so many sequences are kept in shared memory

template <int DP> struct Smem {
  static constexpr int kSlots = DP == 128 ? 5 : 8;
  static constexpr int kTile = kKeys * DP * 2;      // bytes of a K or V tile, and of half the queries
  static constexpr int kBars = (2 + kSlots) * kTile;
  // barriers: two a slot, then queries 2, scores 2, weights 4, queue, drain
  static constexpr int kBarBytes = 8 * (2 * kSlots + 8 + 2 * kQueue + 1);
  static constexpr int kFlags = kBars + (kBarBytes + 63) / 64 * 64;
  static constexpr int kSegs = kFlags + 64;
  // the softmaxes' maxima and sums; before the first segment, the scan
  // of the work
  static constexpr int kStats = kSegs + kQueue * 64;
  static constexpr int kSeqs = kStats + 2048;           // q_start, kv_len
  static constexpr int kBytes = kSeqs + 8 * kCachedSeqs + 16;
  static_assert(kBytes <= 232448, "227 KB a block");
  static_assert(kQueue * sizeof(Segment) <= 256 && kFlags % 16 == 0, "regions");
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

// One lane of the (converged) warp, the same every time.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is;
}

// The MMAs and commits of one warp: every lane computes the operands, so that
// they stay in uniform registers, and the elected one (`lead`) issues. (Issued
// from a branch of one lane, an MMA measured 80 to 115 cycles of its thread,
// more than the 64 it runs.)
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(bar), "r"(lead)
      : "memory");
}

// 128 columns of this thread's TMEM lane -> registers.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&a)[64], float (&b)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
      "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%129];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]),
        "=f"(a[7]), "=f"(a[8]), "=f"(a[9]), "=f"(a[10]), "=f"(a[11]), "=f"(a[12]), "=f"(a[13]),
        "=f"(a[14]), "=f"(a[15]), "=f"(a[16]), "=f"(a[17]), "=f"(a[18]), "=f"(a[19]),
        "=f"(a[20]), "=f"(a[21]), "=f"(a[22]), "=f"(a[23]), "=f"(a[24]), "=f"(a[25]),
        "=f"(a[26]), "=f"(a[27]), "=f"(a[28]), "=f"(a[29]), "=f"(a[30]), "=f"(a[31]),
        "=f"(a[32]), "=f"(a[33]), "=f"(a[34]), "=f"(a[35]), "=f"(a[36]), "=f"(a[37]),
        "=f"(a[38]), "=f"(a[39]), "=f"(a[40]), "=f"(a[41]), "=f"(a[42]), "=f"(a[43]),
        "=f"(a[44]), "=f"(a[45]), "=f"(a[46]), "=f"(a[47]), "=f"(a[48]), "=f"(a[49]),
        "=f"(a[50]), "=f"(a[51]), "=f"(a[52]), "=f"(a[53]), "=f"(a[54]), "=f"(a[55]),
        "=f"(a[56]), "=f"(a[57]), "=f"(a[58]), "=f"(a[59]), "=f"(a[60]), "=f"(a[61]),
        "=f"(a[62]), "=f"(a[63]), "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]),
        "=f"(b[5]), "=f"(b[6]), "=f"(b[7]), "=f"(b[8]), "=f"(b[9]), "=f"(b[10]), "=f"(b[11]),
        "=f"(b[12]), "=f"(b[13]), "=f"(b[14]), "=f"(b[15]), "=f"(b[16]), "=f"(b[17]),
        "=f"(b[18]), "=f"(b[19]), "=f"(b[20]), "=f"(b[21]), "=f"(b[22]), "=f"(b[23]),
        "=f"(b[24]), "=f"(b[25]), "=f"(b[26]), "=f"(b[27]), "=f"(b[28]), "=f"(b[29]),
        "=f"(b[30]), "=f"(b[31]), "=f"(b[32]), "=f"(b[33]), "=f"(b[34]), "=f"(b[35]),
        "=f"(b[36]), "=f"(b[37]), "=f"(b[38]), "=f"(b[39]), "=f"(b[40]), "=f"(b[41]),
        "=f"(b[42]), "=f"(b[43]), "=f"(b[44]), "=f"(b[45]), "=f"(b[46]), "=f"(b[47]),
        "=f"(b[48]), "=f"(b[49]), "=f"(b[50]), "=f"(b[51]), "=f"(b[52]), "=f"(b[53]),
        "=f"(b[54]), "=f"(b[55]), "=f"(b[56]), "=f"(b[57]), "=f"(b[58]), "=f"(b[59]),
        "=f"(b[60]), "=f"(b[61]), "=f"(b[62]), "=f"(b[63])
      : "r"(taddr), "r"(taddr + 64)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Registers a thread: the two softmax warpgroups take what the third one
// leaves (2 x 224 + 56 = 3 x 168, what the block was launched with).
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
}
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}

// 16 bytes from global to shared memory, in the background; zeros if !use.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool use) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(use ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Minus infinity into the scores n of a 64-key piece above hi, or up to lo.
__device__ __forceinline__ void mask_above(float (&s)[64], int hi) {
#pragma unroll
  for (int n = 0; n < 64; ++n) s[n] = n > hi ? -INFINITY : s[n];
}
__device__ __forceinline__ void mask_to(float (&s)[64], int lo) {
#pragma unroll
  for (int n = 0; n < 64; ++n) s[n] = n <= lo ? -INFINITY : s[n];
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
__device__ __forceinline__ float max64(const float (&s)[64]) {
  float a = s[0], b = s[1], c = s[2], d = s[3];
#pragma unroll
  for (int n = 4; n + 8 <= 60; n += 8) {
    a = max3(a, s[n], s[n + 1]);
    b = max3(b, s[n + 2], s[n + 3]);
    c = max3(c, s[n + 4], s[n + 5]);
    d = max3(d, s[n + 6], s[n + 7]);
  }
  a = max3(a, s[60], s[61]);
  b = max3(b, s[62], s[63]);
  return fmaxf(max3(a, b, c), d);
}

// Weights of 64 scores, 2^(scale s + ref), packed in pairs of T into TMEM;
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

__device__ __forceinline__ int64_t scan_warp(int64_t x, int lane) {
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_chunk_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, int numbers) {
  using S = Smem<DP>;
  constexpr int kSlots = S::kSlots, kSub = DP / 64;
  extern __shared__ __align__(1024) uint8_t basep[];
  const uint32_t base = smem_u32(basep);
  if (base & 1023u) {   // the swizzled tiles need it, and there is no room to align
    pdl_wait_primary();
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
      *p.status = kDevTimeout;
      static_cast<CutTile*>(p.cuts)[blockIdx.x] = {};   // nothing to join
    }
    return;
  }
  // queries of the two softmaxes, then the ring, then the barriers
  const uint32_t ring = base + 2 * S::kTile;
  const uint32_t full = base + S::kBars, empty = full + 8 * kSlots, q_full = empty + 8 * kSlots;
  const uint32_t s_full = q_full + 16, p_ready = s_full + 16, seg_full = p_ready + 32;
  const uint32_t seg_empty = seg_full + 8 * kQueue, drain = seg_empty + 8 * kQueue;
  static_assert(S::kBarBytes == 8 * (2 * kSlots) + 16 + 16 + 32 + 16 * kQueue + 8, "barriers");
  volatile uint32_t* const flags = reinterpret_cast<volatile uint32_t*>(basep + S::kFlags);
  volatile uint32_t* const failed = flags + 1;   // flags[0]: TMEM address
  Segment* const queue = reinterpret_cast<Segment*>(basep + S::kSegs);
  int64_t* const scan = reinterpret_cast<int64_t*>(basep + S::kStats);
  Start* const start = reinterpret_cast<Start*>(scan + 20);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool stalled = p.stall_ns > 0 && blockIdx.x == 0;
  const uint64_t limit = stalled ? p.stall_ns : kWaitNs;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbarrier_init(full + 8 * i, 1);
      mbarrier_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbarrier_init(q_full + 8 * i, kSoft / 2);
      mbarrier_init(s_full + 8 * i, 1);
      mbarrier_init(p_ready + 16 * i, 4);       // weights of the first 64 keys
      mbarrier_init(p_ready + 16 * i + 8, 4);   // and of the others
    }
    for (int i = 0; i < kQueue; ++i) {
      mbarrier_init(seg_full + 8 * i, 1);
      mbarrier_init(seg_empty + 8 * i, kSoft / 32 + 2);   // softmax, MMA and TMA warps
    }
    mbarrier_init(drain, 1);
    *failed = 0;
    flags[2] = flags[3] = 0;
    start->number = -1;
    mbarrier_init_fence();
  }
  if (warp == 8) {
    tmem_alloc<1>(smem_u32(const_cast<uint32_t*>(flags)), 512);
    tmem_relinquish<1>();
  }
  pdl_wait_primary();
  pdl_launch_dependents();

  // The block's piece [x0, x1) of the line of work: each thread adds up the
  // cost of some consecutive row tiles of a head, a scan gives the totals.
  int32_t* const seqs = reinterpret_cast<int32_t*>(basep + S::kSeqs);
  const bool cached = p.nseq <= kCachedSeqs;
  if (cached) {
    if ((int)threadIdx.x <= p.nseq) seqs[threadIdx.x] = p.q_start[threadIdx.x];
    if ((int)threadIdx.x < p.nseq) seqs[kCachedSeqs + 1 + threadIdx.x] = p.kv_len[threadIdx.x];
    __syncthreads();
  }
  const Tiles<AttnParams> tiles{p, cached ? seqs : p.q_start, cached ? seqs + kCachedSeqs + 1 : p.kv_len};
  const int per = (numbers + kThreads - 1) / kThreads;
  const int i0 = min((int)threadIdx.x * per, numbers), i1 = min(i0 + per, numbers);
  const int b0 = i0 < i1 ? tiles.find(i0) : 0;
  const int64_t mine = sum_tiles(tiles, numbers, i0, i1, b0);
  int64_t before = scan_warp(mine, lane);
  if (lane == 31) scan[warp] = before;
  before -= mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) before += total;
    total += scan[w];
  }
  const uint32_t tmem = flags[0];
  // What the scheduling warp needs goes through shared memory: held in
  // registers across the roles it was spilled, and its first segment late.
  Start here;
  const int heads = p.q_heads / p.group;
  if (find_start(before, mine, total, numbers, i0, b0, heads, blockIdx.x, gridDim.x, &here)) *start = here;
  // Whether the lengths are what they should be, from the last warp on: the
  // first ones are likelier to find the start.
  for (int b = kThreads - 1 - (int)threadIdx.x; b < p.nseq; b += kThreads) {
    const bool disorder = !tiles.in_order(b);
    if (disorder) flags[3] = 1;   // no work
    if (blockIdx.x == 0 && (disorder || tiles.start(b + 1) - tiles.start(b) > p.max_q ||
                            tiles.kv_len[b] > p.max_positions))
      *p.status = kDevIndex;
  }
  __syncthreads();

  // Every wait has a limit. One that gave up sets `failed`, which ends the
  // other waits too; the warps then run through the rest without waiting (the
  // softmax warps still meet at their barriers), results are undefined and the
  // status word says so. The waits for the segment queue are apart: they only
  // depend on warps that always get there, and all warps see every segment.
  auto wait_for = [&](uint32_t bar, uint32_t parity, uint64_t most, bool heed) {
    if (mbarrier_test_wait(bar, parity)) return true;
    const uint64_t t = global_timer_ns();
    for (uint32_t i = 0; i < (1u << 28) && !(heed && *failed); ++i) {
      if (mbarrier_try_wait(bar, parity)) return true;
      if ((i & 15u) == 15u && global_timer_ns() - t > most) break;
    }
    *failed = 1;
    return false;
  };
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_for(bar, parity, limit, true); };
  auto wait_item = [&](int item) { return wait(full + 8 * (item % kSlots), (item / kSlots) & 1); };
  // The next segment of the queue, for a warp; false at the end.
  auto next_segment = [&](int sg, Segment& g) {
    const bool ok = wait_for(seg_full + 8 * (sg % kQueue), (sg / kQueue) & 1, 20 * kWaitNs, false);
    if (__any_sync(0xffffffffu, !ok)) return false;
    g = queue[sg % kQueue];
    __syncwarp();
    if (lane == 0) mbarrier_arrive(seg_empty + 8 * (sg % kQueue));
    return g.n >= 0;
  };

  // Each role is a loop of its own over the segments (the items of a segment
  // in the ring: K of key tile j is base_item + 2 j, V the one after).
  if (warp < kSoft / 32) {
    registers_up();
    // -------------------------------------------------- softmax
    const int h = warp >> 2, r = threadIdx.x & (kHalf - 1);        // softmax h, row r
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lanes + h * kKeys;            // scores; the weights go over their first half
    const uint32_t to = lanes + 256 + h * DP;         // output
    const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);
    const uint64_t scale2 = f2_packf(scale, scale);
    // Key tiles of segment s for this softmax.
    auto tiles_of = [&](const Segment& s) {
      return s.n < 0 ? 0 : s.rows <= kHalf ? (s.n - h + 1) / 2 : s.n;
    };
    // x / group for row numbers of a tile, by the reciprocal
    auto by_group = [&](int x) {
      return p.group_inv ? (int)__umulhi((uint32_t)x, p.group_inv) : x / p.group;
    };
    // This softmax's 128 rows of queries of segment s, in the background: rows
    // past the end and values past the head are zeros, and all of them with a
    // scale of zero.
    auto load_queries = [&](const Segment& s) {
      if (tiles_of(s) == 0) return;
      const bool alt = s.rows <= kHalf;
      // 16-byte chunk c of every kStep-th row
      constexpr int kStep = kHalf / (DP / 8);
      const int c = r % (DP / 8), qr0 = r / (DP / 8), half = alt ? 0 : h * kHalf;
      const T* const q = static_cast<const T*>(p.q) + (int64_t)s.tok * p.q_stride +
                         (int64_t)s.head * p.group * p.dim + c * 8;
      const bool real = c * 8 < p.dim && p.scale_log2 != 0.0f;
      // (a short loop: its instructions are fetched when the block starts)
#pragma unroll 2
      for (int i = 0; i < kHalf / kStep; ++i) {
        const int qr = qr0 + i * kStep, x = s.off + half + qr;
        const int t = by_group(x), hh = x - t * p.group;
        const bool use = real && half + qr < s.rows;
        copy16(base + h * S::kTile + (c >> 3) * kHalf * 128 + swz(qr, c & 7),
               use ? q + (int64_t)t * p.q_stride + hh * p.dim : p.q, use);
      }
    };
    auto queries_loaded = [&](const Segment& s) {
      if (tiles_of(s) == 0) return;
      copy16_wait();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbarrier_arrive(q_full + 8 * h);
    };
    int base_item = 0;
    uint32_t ss = 0;                                  // scores seen so far
    Segment g;
    for (int sg = 0; next_segment(sg, g); ++sg) {
      // alternate key tiles of the same rows, or the same key tiles of two halves
      const bool alt = g.rows <= kHalf;
      const int row = alt ? r : h * kHalf + r;        // of the row tile
      const int n = tiles_of(g);
      if (sg == 0) {
        load_queries(g);
        queries_loaded(g);
      }
      // the next segment's queries, as soon as this one's are done with
      auto next_queries = [&]() {
        if (wait_for(seg_full + 8 * ((sg + 1) % kQueue), ((sg + 1) / kQueue) & 1, 20 * kWaitNs, false))
          load_queries(queue[(sg + 1) % kQueue]);
      };
      const int trow = by_group(g.off + min(row, g.rows - 1));
      const int pos = g.pos + trow;
      float m = -INFINITY;
      uint64_t l0 = 0, l1 = 0;
      for (int k = 0; k < n; ++k) {
        wait(s_full + 8 * h, ss & 1);
        ++ss;
        if (k == n - 1) next_queries();
        __syncwarp();   // lanes leave a wait apart; tensor memory is read by whole warps
        tc_fence_after();
        const int j = alt ? 2 * k + h : k;
        const int key0 = (g.t0 + j) * kKeys;
        float a[64], b[64];
        tmem_ld128(ts, a, b);
        // the row sees the keys (pos - window, pos]: where the tile has keys past
        // its first row's, or before its last row's window
        if (key0 + kKeys - 1 > g.pos) {
          mask_above(a, pos - key0);
          mask_above(b, pos - key0 - 64);
        }
        if (p.window > 0 && key0 < g.lo + (g.hi - 1 - g.pos)) {
          const int to_key = max(pos - p.window - key0, -1);
          mask_to(a, to_key);
          mask_to(b, to_key - 64);
        }
        const float top = fmaxf(max64(a), max64(b)) * scale;
        if (__any_sync(0xffffffffu, top > m + kGrow || (m == -INFINITY && top > m))) {
          const float mn = fmaxf(m, top);
          const float corr = exp2_approx(m - (mn == -INFINITY ? 0.0f : mn));
          m = mn;
          const uint64_t c2 = f2_packf(corr, corr);
          l0 = f2_mul(l0, c2);
          l1 = f2_mul(l1, c2);
          if (k > 0) {
#pragma unroll
            for (int c = 0; c < DP; c += 32) {
              uint32_t o[32];
              tmem_ld32(to + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tmem_st32(to + c, o);
            }
          }
        }
        // values of keys that no row sees may be anything: zero them (their
        // weights are zero, but zero times NaN is not); both softmaxes do, as
        // neither's product waits for the other
        if (key0 + kKeys > g.hi || key0 < g.lo) {
          const int item = base_item + 2 * j + 1;
          wait_item(item);
          const int key = key0 + r;
          if (key >= g.hi || key < g.lo) {
            uint8_t* v = basep + (2 + item % kSlots) * S::kTile;
#pragma unroll
            for (int c = 0; c < DP / 8; ++c)
              *reinterpret_cast<uint4*>(v + (c >> 3) * kKeys * 128 + swz(r, c & 7)) =
                  make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          named_barrier_sync(2 + h, kHalf);   // all rows, before the first product
        }
        const float ref = addend<T, kUp>(m == -INFINITY ? 0.0f : m);
        const uint64_t ref2 = f2_packf(ref, ref);
        auto signal = [&](uint32_t bar) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbarrier_arrive(bar);
        };
        weights64<T>(a, scale2, ref2, l0, l1, ts);
        signal(p_ready + 16 * h);
        weights64<T>(b, scale2, ref2, l0, l1, ts + 32);
        signal(p_ready + 16 * h + 8);
      }
      if (n > 0) {   // the last product
        wait(s_full + 8 * h, ss & 1);
        ++ss;
      }
      base_item += 2 * g.n;
      if (n == 0) next_queries();
      __syncwarp();
      tc_fence_after();
      queries_loaded(queue[(sg + 1) % kQueue]);
      const float2 la = f2_unpack(f2_add(l0, l1));
      float l = la.x + la.y;
      m -= Scaled<T, kUp>::kUp;
      float keep = 1.0f, other = 0.0f;
      const bool merge = alt && g.n > 1;
      if (merge) {
        // each softmax takes the other one's result from TMEM: warps of the
        // same quadrant reach the same lanes
        float* const stats = reinterpret_cast<float*>(basep + S::kStats);
        stats[2 * h * kHalf + r] = m;
        stats[(2 * h + 1) * kHalf + r] = l;
        tc_fence_before();
        named_barrier_sync(1, kSoft);
        tc_fence_after();
        const float m1 = stats[(2 - 2 * h) * kHalf + r], l1 = stats[(3 - 2 * h) * kHalf + r];
        const float mn = fmaxf(m, m1), ref = mn == -INFINITY ? 0.0f : mn;
        keep = exp2_approx(m - ref);
        other = exp2_approx(m1 - ref);
        l = l * keep + l1 * other;
        m = mn;
      }
      if (merge || !alt || h == 0) {
        // -------------------------------------------- output rows
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float lse = l == 0.0f ? -INFINITY : m + log2f(l);
        const bool live = row < g.rows;
        const int64_t tok = g.tok + trow;
        const int qh = g.head * p.group + (g.off + row) % p.group;
        const int64_t at = (int64_t)g.part * kRows + row;
        if (live && (h == 0 || !alt)) {
          if (g.part >= 0) p.part_lse[at] = lse;
          else if (p.lse) p.lse[tok * p.q_heads + qh] = lse * kLn2;
        }
        void* const out = g.part >= 0 ? static_cast<void*>(p.part_o) : p.o;
        const int type = g.part >= 0 ? TQ_F32 : p.o_type;
        const int64_t obase = g.part >= 0 ? at * p.dim : tok * p.o_stride + (int64_t)qh * p.dim;
        keep *= inv;
        other *= inv;
        // of merged rows each softmax writes half of the values
        const int c0 = merge ? h * (DP / 2) : 0, c1 = merge ? c0 + DP / 2 : DP;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t o[32] = {}, o1[32] = {};
          if (n > 0) tmem_ld32(to + c, o);
          if (merge) tmem_ld32(to + (h == 0 ? DP : -DP) + c, o1);
#pragma unroll
          for (int q = 0; q < 32; q += 16) {
            const int left = p.dim - c - q;
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              x[e] = __uint_as_float(o[q + e]) * keep;
              if (merge) x[e] = fmaf(__uint_as_float(o1[q + e]), other, x[e]);
            }
            if (live && left > 0) store_out16(out, type, obase + c + q, x, left);
          }
          __syncwarp();   // before the next columns, which the warp reads together
        }
      }
      tc_fence_before();
      if (merge) named_barrier_sync(1, kSoft);
    }
  } else {
    registers_down();
    if (warp == 11) {
      // ------------------------------------------------ scheduling
      if (lane == 0) {
        int queued = 0;
        auto push = [&](const Segment& g) {
          const int i = queued % kQueue;
          if (queued >= kQueue)
            wait_for(seg_empty + 8 * i, (queued / kQueue - 1) & 1, 20 * kWaitNs, false);
          queue[i] = g;
          mbarrier_arrive(seg_full + 8 * i);
          ++queued;
        };
        Start st = *start;
        if (flags[3]) st.number = -1;
        const CutTile cut = walk(tiles, numbers, st, p.q_heads / p.group, (int)gridDim.x, (int)blockIdx.x,
                                 push, [&]() { return *failed != 0; });
        Segment end = {};
        end.n = -1;
        push(end);
        static_cast<CutTile*>(p.cuts)[blockIdx.x] = cut;
      }
      __syncwarp();
    } else if (warp == 10) {
      int base_item = 0;
      Segment g;
      for (int sg = 0; next_segment(sg, g); ++sg) {
        // ---------------------------------------------- TMA
        if (__any_sync(0xffffffffu, *failed) || stalled) continue;
        const int boxes = kKeys / p.box_rows;   // 1 .. 16, one lane each
        const int off = lane * p.box_rows;
        bool bad = false;
        // the table's entry for this lane's box of the next tile is loaded a
        // tile ahead and looked at when its turn comes
        int entry = -1, pslot = 0;
        bool seen = false;   // some row sees the box
        auto locate = [&](int t) {
          const int key = t * kKeys + off;
          seen = lane < boxes && t < g.t0 + g.n && key < g.hi && key + p.box_rows > g.lo;
          if (seen) {
            const int lp = key / p.page_size;
            pslot = key - lp * p.page_size;
            entry = lp < p.table_width ? p.table[g.seq * p.table_stride + lp] : -1;
          }
        };
        locate(g.t0);
        for (int j = 0; j < g.n; ++j) {
          // the page one past the cache (zeros, nothing read) for a box that no
          // row sees
          int pg = p.pages, sl = 0;
          if (seen) {
            if (entry >= 0 && entry < p.pages) {
              pg = entry;
              sl = pslot;
            } else {
              bad = true;
            }
          }
          locate(g.t0 + j + 1);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int it = base_item + 2 * j + v, sidx = it % kSlots;
            // (one answer for the warp)
            if (!__all_sync(0xffffffffu, it < kSlots || wait(empty + 8 * sidx, (it / kSlots - 1) & 1))) break;
            if (lane == 0) mbarrier_arrive_expect_tx(full + 8 * sidx, S::kTile);
            __syncwarp();
            if (lane < boxes) {
              const uint32_t dst = ring + sidx * S::kTile + off * 128;
#pragma unroll
              for (int c = 0; c < kSub; ++c)
                tma_box(dst + c * kKeys * 128, v ? &vmap : &kmap, c * 64, sl, g.head, pg,
                        full + 8 * sidx);
            }
            if (lane == 0) flags[2] = it + 1;   // copies issued, for the failure path
          }
          if (__any_sync(0xffffffffu, *failed)) break;
        }
        if (bad) *p.status = kDevIndex;
        base_item += 2 * g.n;
      }
    } else if (warp == 8) {
      int base_item = 0;
      uint32_t qs[2] = {0, 0}, ps[2] = {0, 0};   // queries and weights seen so far
      const uint32_t mtmem = __shfl_sync(0xffffffffu, tmem, 0), lead = elect_one();
      // a negative scale turns S (bit 13 negates A), so that the maximum of S
      // is that of the scores
      const uint32_t idesc_s = Desc<T, DP>::kScores | (p.scale_log2 < 0.0f ? 1u << 13 : 0u);
      constexpr uint32_t idesc_o = Desc<T, DP>::kOut;
      Segment g;
      for (int sg = 0; next_segment(sg, g); ++sg) {
        // ---------------------------------------------- MMA
        // One warp for both softmaxes, in turn: with a warp for each, the two
        // fall into step, both computing weights and then both waiting for
        // products (1372 us where this order takes 1150).
        const int n = __shfl_sync(0xffffffffu, g.n, 0);
        const bool alt = __shfl_sync(0xffffffffu, g.rows, 0) <= kHalf;
        auto qk = [&](int h, int item) {
          const uint64_t a = desc_k(base + h * S::kTile), b = desc_k(ring + (item % kSlots) * S::kTile);
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) {
            const uint64_t o = ((d >> 2) * kKeys * 128 + (d & 3) * 32) >> 4;
            mma_ss(lead, mtmem + h * kKeys, a + o, b + o, idesc_s, d > 0);
          }
        };
        auto pv = [&](int h, int item, int part, bool first) {
          const uint64_t b = desc_n(ring + (item % kSlots) * S::kTile);
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) {
            const int k = part * (kKeys / 32) + i;
            mma_ts(lead, mtmem + 256 + h * DP, mtmem + h * kKeys + k * 8, b + k * (2048 >> 4), idesc_o,
                   !(first && k == 0));
          }
        };
        auto free_slot = [&](int item) { commit(lead, empty + 8 * (item % kSlots)); };
        // all lanes wait; one that gave up ends it for all
        auto ready = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
        // key tiles of softmax h, and its k-th one
        auto count = [&](int h) { return alt ? (n - h + 1) / 2 : n; };
        auto tile_of = [&](int h, int k) { return alt ? 2 * k + h : k; };
        bool ok = !__any_sync(0xffffffffu, *failed);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (count(h) == 0 || !ok) continue;
          const int ki = base_item + 2 * tile_of(h, 0);
          ok = ready(wait(q_full + 8 * h, qs[h] & 1) && wait_item(ki));
          if (!ok) continue;
          ++qs[h];
          tc_fence_after();
          qk(h, ki);
          commit(lead, s_full + 8 * h);
          if (alt || h == 1) free_slot(ki);
        }
        for (int k = 0; k < count(0) && ok; ++k) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (k >= count(h) || !ok) continue;
            const int vi = base_item + 2 * tile_of(h, k) + 1;
            const int ki = base_item + 2 * tile_of(h, k + 1);
            // the second half's tiles are there: the first one waited for them
            const bool own = alt || h == 0;
            ok = ready((!own || wait_item(vi)) && wait(p_ready + 16 * h, ps[h] & 1));
            if (!ok) continue;
            tc_fence_after();
            pv(h, vi, 0, k == 0);
            ok = ready(wait(p_ready + 16 * h + 8, ps[h] & 1));
            if (!ok) continue;
            ++ps[h];
            tc_fence_after();
            pv(h, vi, 1, k == 0);
            if (k + 1 < count(h)) {
              if (own) ok = ready(wait_item(ki));
              if (!ok) continue;
              qk(h, ki);
            }
            commit(lead, s_full + 8 * h);
            if (alt || h == 1) {
              free_slot(vi);
              if (k + 1 < count(h)) free_slot(ki);
            }
          }
        }
        base_item += 2 * n;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();   // no wait of a role runs out after it
  tc_fence_after();
  if (*failed) {
    // no block leaves before its copies have landed and its MMAs have ended
    if (warp == 10) {
      const int issued = (int)flags[2];
      const int last = lane < kSlots ? last_phase(issued, lane, kSlots) : -1;
      if (last >= 0) mbarrier_wait_bounded(full + 8 * lane, last, limit / 10);
    }
    if (warp == 8) {
      commit(elect_one(), drain);
      mbarrier_wait_bounded(drain, 0, limit / 10);
    }
    if (threadIdx.x == 0) *p.status = kDevTimeout;
    __syncwarp();
  }
  if (warp == 8) tmem_dealloc<1>(tmem, 512);
}

constexpr int kJoinWarps = 8, kJoinBlocks = 32;  // warps of a block, blocks of a row tile

// Joins the pieces of the row tiles that were cut: o = sum_s 2^(lse_s - M) o_s
// / sum_s 2^(lse_s - M), a warp per row.
__global__ void __launch_bounds__(kJoinWarps * 32)
attn_chunk_join_kernel(const __grid_constant__ AttnParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const CutTile cut = static_cast<const CutTile*>(p.cuts)[blockIdx.x];
  if (cut.n == 0) return;
  const int lane = threadIdx.x & 31;
  for (int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); r < cut.rows; r += kJoinWarps * kJoinBlocks) {
    auto row_of = [&](int i) {
      return (int64_t)(i == 0 ? cut.part0 : 2 * ((int)blockIdx.x + i)) * kRows + r;
    };
    // 32 pieces at a time, a lane's weight for each; their values are loaded
    // beside the weights
    float top = -INFINITY, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < cut.n; i0 += 32) {
      const int n = min(32, cut.n - i0);
      const float lse = lane < n ? p.part_lse[row_of(i0 + lane)] : -INFINITY;
      float4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n && lane * 4 < p.dim)
          x[i] = *reinterpret_cast<const float4*>(p.part_o + row_of(i0 + i) * p.dim + lane * 4);
      float m = lse;
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      m = fmaxf(m, top);
      const float ref = m == -INFINITY ? 0.0f : m, old = exp2_approx(top - ref);
      top = m;
      float w = exp2_approx(lse - ref), all = w;
      for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
      sum = sum * old + all;
      acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
      for (int j = 0; j < n; j += 8) {
        float4 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j + 8 + i < n && lane * 4 < p.dim)
            x[i] = *reinterpret_cast<const float4*>(p.part_o + row_of(i0 + j + 8 + i) * p.dim + lane * 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = __shfl_sync(0xffffffffu, w, (j + i) & 31);
          if (j + i < n && lane * 4 < p.dim) {
            acc.x = fmaf(f, y[i].x, acc.x);
            acc.y = fmaf(f, y[i].y, acc.y);
            acc.z = fmaf(f, y[i].z, acc.z);
            acc.w = fmaf(f, y[i].w, acc.w);
          }
        }
      }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int t = (cut.off + r) / p.group;
    const int64_t tok = cut.tok + t, qh = cut.head * p.group + (cut.off + r - t * p.group);
    const float x[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    if (lane * 4 < p.dim) store_out4(p.o, p.o_type, tok * p.o_stride + qh * p.dim + lane * 4, x);
    if (lane == 0 && p.lse)
      p.lse[tok * p.q_heads + qh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

template <typename T, int DP>
cudaError_t launch_chunk(const AttnParams& p, const AttnCall& c, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, cudaStream_t s) {
  auto kernel = attn_chunk_kernel<T, DP>;
  const cudaError_t e = ensure_dynamic_smem((const void*)kernel, Smem<DP>::kBytes);
  if (e != cudaSuccess) return e;
  DeviceLimits lim;
  cudaError_t r = device_limits(&lim);
  if (r != cudaSuccess) return r;
  const int grid = lim.sms < c.plan.blocks ? lim.sms : c.plan.blocks;
  r = launch_pdl(kernel, dim3(grid), dim3(kThreads), Smem<DP>::kBytes, s, p, kmap, vmap,
                 (int)c.plan.tiles_x);
  if (r != cudaSuccess) return r;
  return launch_pdl(attn_chunk_join_kernel, dim3(grid, kJoinBlocks), dim3(kJoinWarps * 32), 0, s,
                    p);
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
