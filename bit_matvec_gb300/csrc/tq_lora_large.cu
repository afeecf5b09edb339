// tq_lora_large.cu -- low-rank adapters for many tokens each: tiles of 128 tokens on the 5th-generation
// tensor cores.
//
// A cluster of four thread blocks takes a tile: each block a quarter of A's columns for h = A x, the four
// parts summed through distributed shared memory, then each block a quarter of the rows of Y = Z + B h.
// With 128 tokens a tile, A and B are read from L2 a quarter as often as with the 32 of tq_lora.cu; what is left
// for the threads is the traffic itself: x in, Z in, Y out. (Clusters of eight: 273 us where four took 183; the GPU
// holds 15 of them with a block an SM, and 36 of four.)
//
// Ranks above 64 take several passes of 64 over Y, of 32-bit values: a pass adds to what the one before
// has stored, which is the same 32-bit sum. (16-bit Y would be rounded twice: such calls take tq_lora.cu.)
//
// Taken for ranks above 32, at least 4096 tokens and 512 an adapter (a slot, used or not); from 2048 tokens on above
// rank 112, where tq_lora.cu has room for one thread block an SM. us, this kernel and that of tq_lora.cu, f32:
// matrices of 5120 x 15360, rank 64, 4096 tokens of four adapters 158 and 277, of sixteen 251 and 282; 8192 of
// sixteen 348 and 530; 2048 of one 143 and 149; 4096 of two, rank 32, 158 and 177, rank 16 159 and 149; 8192 of
// sixteen, ranks of several sizes up to 32, 17408 rows: 329 and 345. Matrices of 5120 x 5120, 4096 tokens of two:
// rank 45 106 and 200, 100 165 and 279, 128 165 and 417, 256 311 and 751; 2048 tokens of one: rank 64 76 and 90, 100
// 143 and 149, 128 143 and 234; 1024 of one, rank 128: 138 and 137. (The limits are from when this kernel took a
// sixth more: calls of 2048 tokens, or of rank 32, that would be a little faster here still go the other way.)
//
// Products are tcgen05 kind::tf32 with 128 tokens as rows of A, operands in shared memory without a
// swizzle: 16-byte columns (four values of the contraction index), 128 rows of each one after another,
// columns 16 bytes further apart than that, so that threads that write neighbouring columns meet no bank
// twice. x and h are the sum of two tf32 parts, those of x multiplied one after the other into the same accumulator,
// those of h into two that are added by the threads (tq_lora.cuh: infinite weights).
// The first product's columns go to eight accumulators one after the other, which are added in 32 bits: the
// tensor cores cut their sums, which leans one way over many steps. After 16 chunks of 32 columns in each (16384
// columns of the matrix) they are read and begun again. (2^20 columns of one sign, divided among the eight
// however many there are, were 4.0e-4 off; now 6.0e-6.)
//
// A warp takes its 32 tokens' sums of 32 rows from tensor memory, a token a lane, and turns them through
// shared memory into rows of 128 bytes of four tokens at a time, as it has loaded them of Z a tile ahead and
// stores them to Y. (With a token a lane to the end every load and store met 32 lines of the cache.)
//
// What bounds it: at 4096 tokens, 5120 columns, 15360 rows, rank 64, f32, 159 us or 3.7 TB/s. (The offsets of the
// tokens' rows of Y and Z stand in shared memory: in registers 52 bytes a thread were spilled, loads of Z under way
// among them, and it took 183 us, 194 with the parts of h summed apart.) The time goes by whole waves of 36
// clusters: of two adapters these are 33 tiles or so, which leaves some 20 SMs without work; sixteen have about 40
// tiles, a second wave (251 us). Within a tile the eight warps' own loads, turns and stores take turns; the first
// product is a fifth of it. (Sixteen warps, with 96 registers a thread for 168: 229 us where eight took 184.)
#include <algorithm>

#include "tq_lora.cuh"
#include "tq_ring.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;              // eight warps that load, convert and store,
constexpr int kAll = kThreads + 32;        // and one that issues the products
constexpr int kM = kLargeTile;
constexpr int kCluster = 4;                // thread blocks that share a tile
constexpr int N = 64;                      // values of h a token; larger ranks take several passes
constexpr int kLeastRank = 33, kLeastTokens = 4096, kLeastTokensEach = 512;
constexpr int kHighRank = 113, kLeastTokensHigh = 2048;
constexpr int kStages = 3;                 // of 32 columns of x and A in shared memory
constexpr int kRows = 128;                 // rows of Y of a tile of the second product
constexpr int kColumn = kM * 16 + 16;      // bytes of a 16-byte column of 128 rows
constexpr int kAhead = 4;                  // chunks of 32 columns of x and A under way
constexpr int kAccs = 8;                   // accumulators of the first product: 64 columns of TMEM each,
constexpr int kChain = 16;                 // chunks that one of them sums up at most,
constexpr int kRound = kAccs * kChain;     // and all of them until they are read
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 1000000000ull;

constexpr int kXStage = 2 * 8 * kColumn;                   // both parts of 32 columns of x
constexpr int kWStage = 8 * (N * 16 + 16);             // 32 columns of A
constexpr int kHBytes = 2 * (N / 4) * kColumn;         // both parts of h
constexpr int kBBytes = (N / 4) * kColumn;             // 128 rows of B
constexpr int kOffsets = 1024;                         // bytes from Y and Z to the tokens' rows
constexpr int kHead = kOffsets + 2 * kM * 8;
constexpr int kUnion = std::max(kStages * (kXStage + kWStage), kHBytes + 2 * kBBytes);
constexpr int kPartPitch = N + 4;                      // floats
constexpr int kTurnPitch = 36;                             // floats of a token's 32 sums on their way to rows
constexpr int kTurn = kThreads * kTurnPitch * 4;
constexpr int kPart = std::max(kM * kPartPitch * 4, kTurn);    // (the parts of h make room for them)
constexpr int kSlice = kM / kCluster * kPartPitch * 4;
constexpr int kSmem = kHead + kUnion + kPart + kSlice;
static_assert(kSmem <= 227 * 1024, "shared memory of a block");
static_assert(kRound % kAhead == 0, "rounds of whole turns");

// kind::tf32: D f32, A and B tf32 (format 2), both K-major.
__device__ __forceinline__ uint32_t idesc_tf32(int m, int n) {
  return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_tf32_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void put16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void split4(const uint4& v, uint4& hi, uint4& lo) {
  split(__uint_as_float(v.x), hi.x, lo.x);
  split(__uint_as_float(v.y), hi.y, lo.y);
  split(__uint_as_float(v.z), hi.z, lo.z);
  split(__uint_as_float(v.w), hi.w, lo.w);
}

// Loads from tensor memory are over; their values are named, so that none is used before.
__device__ __forceinline__ void wait_loads(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
}

template <typename TX, typename TW>
__global__ void __launch_bounds__(kAll, 1) lora_large_kernel(const __grid_constant__ LoraArgs p) {
  constexpr bool kSplit = sizeof(TX) == 4;
  constexpr int kXPieces = kSplit ? 4 : 2;          // 16-byte pieces of a chunk of x a thread
  constexpr int kWColumn = N * 16 + 16;
  extern __shared__ __align__(1024) unsigned char smem[];
  int* const s_tok = reinterpret_cast<int*>(smem);                    // [kM]
  // stages filled and read of the first product; B's buffers filled, and products done, of the second
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + 512);     // [kStages]
  uint64_t* const read = full + kStages;                              // [kStages]
  uint64_t* const b_full = read + kStages;                            // [2]
  uint64_t* const done = b_full + 2;                                  // [2]
  uint64_t* const never = done + 2;          // test facility: nothing arrives here
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + 640);
  int64_t* const s_y = reinterpret_cast<int64_t*>(smem + kOffsets);   // [kM], -1: no such token
  int64_t* const s_z = s_y + kM;                                      // [kM]
  const uint32_t base = smem_u32(smem + kHead);
  float* const part = reinterpret_cast<float*>(smem + kHead + kUnion);
  float* const slice = reinterpret_cast<float*>(smem + kHead + kUnion + kPart);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t crank = cluster_rank();
  const int want = blockIdx.x / kCluster;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int ntiles = *p.ntiles;
  const int4 tile = p.tiles[want];        // adapter, rank, first of order, tokens
  if (want >= ntiles) return;
  const int count = tile.w, rank = min(N, max(0, tile.y - p.rank_from));
  if (p.rank_from > 0 && rank == 0) return;
  const int bytes = p.y_type == TQ_F32 ? 4 : 2;
  if (tid < kM) {
    const int64_t token = tid < count ? p.order[tile.z + tid] : 0;
    s_tok[tid] = (int)token;
    s_y[tid] = tid < count ? token * p.y_stride * bytes : -1;
    s_z[tid] = tid < count ? token * p.z_stride * bytes : -1;
  }
  // rows of B and Y of this thread block, from a multiple of 32 on
  const int rows = (int)p.l.rows, units = (rows + 31) / 32, share = (int)crank;
  const int begin = (int)((int64_t)units * share / kCluster) * 32;
  const int end = min(rows, (int)((int64_t)units * (share + 1) / kCluster) * 32);
  if (tile.x < 0) {
    __syncthreads();
    copy_rows(p, s_tok, count, begin, max(0, end - begin), kAll);
    return;
  }
  const bool issuer = warp == kThreads / 32;
  if (issuer) {
    tc::tmem_alloc<1>(smem_u32(tmem_slot), kTmemCols);
    tc::tmem_relinquish<1>();
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbarrier_init(smem_u32(full + i), kThreads / 32);
      mbarrier_init(smem_u32(read + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbarrier_init(smem_u32(b_full + i), kThreads / 32);
      mbarrier_init(smem_u32(done + i), 1);
    }
    mbarrier_init(smem_u32(never), 1);
    mbarrier_init_fence();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool failed = false;
  // (The test's limit is read where a wait is not over at once: kept in registers it was spilled for. For the
  // same reason it is the one thread that issues the products that stalls.)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!failed && !mbarrier_try_wait(smem_u32(bar), parity)) {
      const uint64_t stall = blockIdx.x == 0 ? p.stall_ns : 0;
      if (!mbarrier_wait_bounded(smem_u32(bar), parity, stall > 0 ? stall : kWaitLimitNs)) failed = true;
    }
  };
  // what this warp's threads have stored to shared memory, for the tensor cores
  auto hand_over = [&](uint64_t* bar) {
    fence_async();
    __syncwarp();
    if (lane == 0) mbarrier_arrive(smem_u32(bar));
  };

  // ---- h = A x over this block's columns, 32 at a time
  const int cols = (int)p.l.cols, chunks = (cols + 31) / 32;
  const int chunk0 = (int)((int64_t)chunks * crank / kCluster), chunk1 = (int)((int64_t)chunks * (crank + 1) / kCluster);
  const int nk = chunk1 - chunk0;
  const int tiles = max(0, (end - begin + kRows - 1) / kRows);
  const uint32_t hs = base, bs = base + kHBytes;
  constexpr int kQuads = N / 4;
  if (issuer) {
    // ---- the products, by one thread
    const bool stalled = p.stall_ns > 0 && blockIdx.x == 0;
    if (lane == 0) {
      const uint32_t idesc1 = idesc_tf32(kM, N), idesc2 = idesc_tf32(kM, kRows);
      for (int k = 0, stage = 0, phase = 0; k < nk; ++k) {
        wait(stalled ? never : full + stage, stalled ? 0 : phase);
        tc::tc_fence_after();
        const uint32_t xs = base + stage * (kXStage + kWStage), ws = xs + kXStage;
        const int in_round = k % kRound, round = max(min(nk - (k - in_round), kRound), kAccs);
        const int acc = in_round * kAccs / round;
        const uint32_t d = tmem + acc * N;
        const bool fresh = in_round == 0 || (in_round - 1) * kAccs / round != acc;
        if (!failed) {
#pragma unroll
          for (int h = 0; h < (kSplit ? 2 : 1); ++h)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_tf32_ss(d, tc::smem_desc(xs + (8 * h + 2 * kk) * kColumn, kColumn, 128),
                          tc::smem_desc(ws + 2 * kk * kWColumn, kWColumn, 128), idesc1,
                          fresh && h == 0 && kk == 0 ? 0u : 1u);
        }
        tc::mma_commit(smem_u32(read + stage));     // (also on failure: it keeps the others' phases moving)
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
    if (lane == 0) {
      const uint32_t idesc2 = idesc_tf32(kM, kRows);
      for (int i = 0; i < tiles; ++i) {
        wait(stalled ? never : b_full + (i & 1), stalled ? 0 : (i >> 1) & 1);
        tc::tc_fence_after();
        const uint32_t d = tmem + (i & 1) * 2 * kRows, b = bs + (i & 1) * kBBytes;
        if (!failed) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int kk = 0; kk < N / 8; ++kk)
              mma_tf32_ss(d + h * kRows, tc::smem_desc(hs + (h * kQuads + 2 * kk) * kColumn, kColumn, 128),
                          tc::smem_desc(b + 2 * kk * kColumn, kColumn, 128), idesc2, kk == 0 ? 0u : 1u);
        }
        tc::mma_commit(smem_u32(done + (i & 1)));
      }
    }
    __syncwarp();
  } else {
  // x: a row's pieces of 16 bytes are neighbouring lanes'; A: a row a quad
  constexpr int kLanes = kSplit ? 8 : 4, kRowsAtOnce = 32 / kLanes;
  const int xc = lane % kLanes, xr = warp * 16 + lane / kLanes;
  const int wr = tid >> 2, wt = tid & 3;
  const TX* from_x[kXPieces];
#pragma unroll
  for (int i = 0; i < kXPieces; ++i) {
    const int row = xr + i * kRowsAtOnce;
    from_x[i] = row < count ? static_cast<const TX*>(p.x) + s_tok[row] * p.x_stride + chunk0 * 32 + xc * (16 / (int)sizeof(TX))
                            : nullptr;
  }
  const TW* const from_w = static_cast<const TW*>(p.l.a) + tile.x * p.l.a_stride + (p.rank_from + wr) * p.l.a_row_stride + chunk0 * 32 + 8 * wt;
  uint4 xv[kAhead][kXPieces], wv[kAhead];
  auto load = [&](int k, uint4 (&x)[kXPieces], uint4& w) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int at = (chunk0 + k) * 32;
#pragma unroll
    for (int i = 0; i < kXPieces; ++i)
      x[i] = k < nk && from_x[i] && at + xc * (16 / (int)sizeof(TX)) < cols
                 ? ldg_stream_v4(from_x[i] + k * 32) : zero;
    w = k < nk && wr < rank && at + 8 * wt < cols ? __ldg(reinterpret_cast<const uint4*>(from_w + k * 32)) : zero;
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, xv[u], wv[u]);
  // The accumulators of the products of `upto` chunks, and of the rounds before, as this block's part of h: a
  // warp's 32 tokens, a token a lane.
  const int half = warp >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  auto read_accs = [&](int upto) {
    // the last products are done, and with them those before
    if (upto > 0) wait(read + (upto - 1) % kStages, ((upto - 1) / kStages) & 1);
    failed = __any_sync(0xffffffffu, failed);        // (tcgen05.ld takes a whole warp)
    tc::tc_fence_after();
    const int accs = upto > 0 ? min((upto - 1) % kRound + 1, kAccs) : 0;
#pragma unroll 1
    for (int g = half; g < N / 16; g += 2) {
      float* const to = part + row * kPartPitch + g * 16;
      float sum[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) sum[e] = upto > kRound ? to[e] : 0.0f;
      if (!failed)
#pragma unroll 1
        for (int a = 0; a < accs; ++a) {
          uint32_t v[16];
          tc::tmem_ld16_nowait(tmem + lanes + a * N + g * 16, v);
          wait_loads(v);
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[e] += __uint_as_float(v[e]);
        }
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(to + e) = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
    }
    tc::tc_fence_before();
  };
  int stage = 0;
  uint32_t phase = 1;           // of the last reading of a stage: none yet
#pragma unroll 1
  for (int r0 = 0; r0 < nk; r0 += kRound) {
    if (r0 > 0) read_accs(r0);       // (what is handed over next says that it is done)
    const int r1 = min(nk, r0 + kRound);
#pragma unroll 1
    for (int k0 = r0; k0 < r1; k0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u;
        if (k >= nk) break;
        const uint32_t xs = base + stage * (kXStage + kWStage), ws = xs + kXStage;
        if (k >= kStages) wait(read + stage, phase);
#pragma unroll
        for (int i = 0; i < kXPieces; ++i) {
          const uint32_t at = xs + (xr + i * kRowsAtOnce) * 16;
          if constexpr (kSplit) {
            uint4 hi, lo;
            split4(xv[u][i], hi, lo);
            put16(at + xc * kColumn, hi);
            put16(at + (8 + xc) * kColumn, lo);
          } else {
            const uint4 v = xv[u][i];
            uint4 a, b;
            widen<TX>(v.x, a.x, a.y);
            widen<TX>(v.y, a.z, a.w);
            widen<TX>(v.z, b.x, b.y);
            widen<TX>(v.w, b.z, b.w);
            put16(at + 2 * xc * kColumn, a);
            put16(at + (2 * xc + 1) * kColumn, b);
          }
        }
        if (wr < N) {
          const uint4 v = wv[u];
          uint4 a, b;
          widen<TW>(v.x, a.x, a.y);
          widen<TW>(v.y, a.z, a.w);
          widen<TW>(v.z, b.x, b.y);
          widen<TW>(v.w, b.z, b.w);
          put16(ws + 2 * wt * kWColumn + wr * 16, a);
          put16(ws + (2 * wt + 1) * kWColumn + wr * 16, b);
        }
        load(k + kAhead, xv[u], wv[u]);
        hand_over(full + stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  }

  // ---- what the second product starts with, on its way from here on
  constexpr int kRowStep = kThreads / kQuads, kBPieces = kRows / kRowStep;
  const int bq = tid % kQuads, br = tid / kQuads;
  const TW* const B = static_cast<const TW*>(p.l.b) + tile.x * p.l.b_stride + p.rank_from;
  uint2 bv[kBPieces];
  const bool whole_b = p.b_vec && rank % 4 == 0;      // a thread's four values all there, or none
  auto load_b = [&](int n0) {
    const int k = 4 * bq;
    if (whole_b) {
#pragma unroll
      for (int i = 0; i < kBPieces; ++i) {
        const int n = n0 + br + i * kRowStep;
        bv[i] = n < end && k < rank ? __ldg(reinterpret_cast<const uint2*>(B + n * p.l.b_row_stride + k)) : make_uint2(0, 0);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kBPieces; ++i) {
      const int n = n0 + br + i * kRowStep;
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = n < end && k + e < rank
                   ? __ldg(reinterpret_cast<const unsigned short*>(B + n * p.l.b_row_stride + k) + e) : 0u;
      bv[i] = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
    }
  };
  // A warp's tokens and half of a tile's rows of Y. Pieces of 16 bytes: of 32 rows a token has 8 (or 4, of
  // 16-bit types), neighbouring lanes'; a lane's pieces are of every fourth (eighth) token.
  const int first = (warp & 3) * 32;
  const bool f32 = p.y_type == TQ_F32;
  const int in_row = f32 ? lane & 7 : lane & 3, of_token = f32 ? lane >> 3 : lane >> 2;
  const int step = f32 ? 4 : 8, turns = f32 ? 8 : 4, values = 16 / bytes;
  const char* const Z = static_cast<const char*>(p.z);
  char* const Y = static_cast<char*>(p.y);
  uint4 zv[2][8];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < 8; ++i) zv[g][i] = make_uint4(0, 0, 0, 0);
  // of 32 rows: g of the two of this warp's half, in the tile that starts `ahead` rows from begin
  auto load_z = [&](int ahead, int g, uint4 (&z)[8]) {
    const int64_t n = begin + ahead + half * 64 + g * 32 + in_row * values;
    if (!Z || n >= end) return;
    const char* const from = Z + n * bytes;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = i < turns ? s_z[first + of_token + i * step] : -1;
      if (at >= 0) z[i] = *reinterpret_cast<const uint4*>(from + at);
    }
  };
  load_b(begin);
  load_z(0, 0, zv[0]);
  load_z(0, 1, zv[1]);

  // ---- this block's part of h
  read_accs(nk);
  // ---- of the whole: a quarter of the tokens summed by each block, then all of them taken
  cluster_arrive();
  cluster_wait();
  const float scale = p.l.scale ? __ldg(p.l.scale + tile.x) : 1.0f;
  for (int i = tid; i < kM / kCluster * kQuads; i += kThreads) {
    const int j = i / kQuads, q = i % kQuads;
    const uint32_t from = smem_u32(part + ((int)crank * (kM / kCluster) + j) * kPartPitch + 4 * q);
    float4 v[kCluster];
#pragma unroll
    for (int c = 0; c < kCluster; ++c) v[c] = load_remote(from, c);
    float4 h = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      h.x += v[c].x;
      h.y += v[c].y;
      h.z += v[c].z;
      h.w += v[c].w;
    }
    const int of = (int)crank * (kM / kCluster) + j;      // among the tile's tokens
    const float sum = (h.x + h.y) + (h.z + h.w);            // (NaN if one of them is)
    if (kSplit && sum != sum && of < count)
      h = dots_again(h, static_cast<const TX*>(p.x) + s_tok[of] * p.x_stride,
                     static_cast<const TW*>(p.l.a) + tile.x * p.l.a_stride + p.rank_from * p.l.a_row_stride,
                     p.l.a_row_stride, 4 * q, rank, cols);
    *reinterpret_cast<float4*>(slice + j * kPartPitch + 4 * q) =
        make_float4(h.x * scale, h.y * scale, h.z * scale, h.w * scale);
  }
  cluster_arrive();
  cluster_wait();
#pragma unroll 4
  for (int i = tid; i < kM * kQuads; i += kThreads) {
    const int j = i % kM, q = i / kM;
    const float4 v = load_remote(smem_u32(slice + (j % (kM / kCluster)) * kPartPitch + 4 * q), j / (kM / kCluster));
    // (past the rank an infinite activation has left a NaN)
    const uint4 w = make_uint4(4 * q < rank ? __float_as_uint(v.x) : 0u, 4 * q + 1 < rank ? __float_as_uint(v.y) : 0u,
                               4 * q + 2 < rank ? __float_as_uint(v.z) : 0u, 4 * q + 3 < rank ? __float_as_uint(v.w) : 0u);
    uint4 hi, lo;
    split4(w, hi, lo);
    put16(hs + q * kColumn + j * 16, hi);
    put16(hs + (kQuads + q) * kColumn + j * 16, lo);
  }
  cluster_arrive();       // this block's slice has no reader left when all have arrived

  // ---- Y = Z + B h, 128 rows at a time: the products of a tile run while the one before is stored
  auto put_b = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kBPieces; ++i) {
      uint4 v;
      widen<TW>(bv[i].x, v.x, v.y);
      widen<TW>(bv[i].y, v.z, v.w);
      put16(bs + buf * kBBytes + bq * kColumn + (br + i * kRowStep) * 16, v);
    }
  };
  // all of h is in place before any of the products (a warp's share of it is handed over with its B)
  named_barrier_sync(1, kThreads);
  if (tiles > 0) {
    put_b(0);
    hand_over(b_full);
    load_b(begin + kRows);
  }
#pragma unroll 1
  for (int i = 0; i < tiles; ++i) {
    if (i + 1 < tiles) {
      put_b((i + 1) & 1);
      tc::tc_fence_before();       // (the accumulator of two tiles ago is read)
      hand_over(b_full + ((i + 1) & 1));
      load_b(begin + (i + 2) * kRows);
    }
    wait(done + (i & 1), (i >> 1) & 1);
    failed = __any_sync(0xffffffffu, failed);
    tc::tc_fence_after();
    float* const turn = part + warp * 32 * kTurnPitch;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
      for (int c = 0; c < 32; c += 16) {
        uint32_t hi[16], lo[16];
        const uint32_t at = tmem + lanes + (i & 1) * 2 * kRows + half * 64 + g * 32 + c;
        if (!failed) {
          tc::tmem_ld16_nowait(at, hi);
          tc::tmem_ld16_nowait(at + kRows, lo);
          wait_loads(hi);
          wait_loads(lo);
        }
        auto sum = [&](int e) { return joined(__uint_as_float(hi[e]), __uint_as_float(lo[e])); };
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<float4*>(turn + lane * kTurnPitch + c + e) =
              make_float4(sum(e), sum(e + 1), sum(e + 2), sum(e + 3));
      }
      const int ahead = i * kRows;
      __syncwarp();
      const int64_t n = begin + ahead + half * 64 + g * 32 + in_row * values;
      if (!failed && n < end) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t at = u < turns ? s_y[first + of_token + u * step] : -1;
          if (at < 0) continue;
          const float* const from = turn + (of_token + u * step) * kTurnPitch + in_row * values;
          const float4 a = *reinterpret_cast<const float4*>(from);
          const uint4 z = zv[g][u];
          uint4* const to = reinterpret_cast<uint4*>(Y + n * bytes + at);
          if (f32) {
            *to = make_uint4(__float_as_uint(a.x + __uint_as_float(z.x)), __float_as_uint(a.y + __uint_as_float(z.y)),
                             __float_as_uint(a.z + __uint_as_float(z.z)), __float_as_uint(a.w + __uint_as_float(z.w)));
          } else {
            const float4 b = *reinterpret_cast<const float4*>(from + 4);
            auto sum = [&](float x, float y, uint32_t w) {
              return (uint32_t)down(x + up((uint16_t)w, p.y_type), p.y_type) |
                     (uint32_t)down(y + up((uint16_t)(w >> 16), p.y_type), p.y_type) << 16;
            };
            *to = make_uint4(sum(a.x, a.y, z.x), sum(a.z, a.w, z.y), sum(b.x, b.y, z.z), sum(b.z, b.w, z.w));
          }
        }
      }
      __syncwarp();
      load_z(ahead + kRows, g, zv[g]);
    }
  }
  }
  if (failed) atomicExch(p.status, kDevTimeout);
  // Where a wait ran out, products that were issued may still write tensor memory. The thread that issued
  // them waits for each last phase: it alone knows that the phases before were begun, and a wait for the
  // parity of a later one would end at once. (Otherwise all have been waited for, and this takes no time.)
  if (issuer && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      const int last = last_phase(nk, i, kStages);
      if (last >= 0) mbarrier_wait_bounded(smem_u32(read + i), (uint32_t)last, kWaitLimitNs);
    }
    for (int i = 0; i < 2; ++i) {
      const int last = last_phase(tiles, i, 2);
      if (last >= 0) mbarrier_wait_bounded(smem_u32(done + i), (uint32_t)last, kWaitLimitNs);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (issuer) {
    tc::tc_fence_after();
    tc::tmem_dealloc<1>(tmem, kTmemCols);
  }
  cluster_wait();
}

template <typename TX, typename TW> cudaError_t launch_as(const LoraArgs& a, int64_t tiles, cudaStream_t s) {
  const auto kernel = lora_large_kernel<TX, TW>;
  cudaError_t e = ensure_dynamic_smem((const void*)kernel, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t grid = tiles * kCluster;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kAll);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

bool lora_large_fits(const LoraArgs& a, int64_t ntok) {
  return a.l.max_rank >= kLeastRank && (a.l.max_rank <= N || a.y_type == TQ_F32) && ntok >= (a.l.max_rank >= kHighRank ? kLeastTokensHigh : kLeastTokens) &&
         ntok >= kLeastTokensEach * a.l.adapters && a.l.rows % (a.y_type == TQ_F32 ? 4 : 8) == 0 && a.y_vec && a.z_vec;
}

cudaError_t launch_lora_large(const LoraArgs& call, int64_t tiles, int x_type, cudaStream_t s) {
  LoraArgs a = call;
  a.stall_ns = (uint64_t)take_debug_stall();
  cudaError_t e = cudaSuccess;
  for (; a.rank_from < std::max<int64_t>(1, a.l.max_rank) && e == cudaSuccess; a.rank_from += N) {
    if (a.l.type == TQ_F16)
      e = x_type == TQ_F32 ? launch_as<float, __half>(a, tiles, s) : launch_as<__half, __half>(a, tiles, s);
    else
      e = x_type == TQ_F32 ? launch_as<float, __nv_bfloat16>(a, tiles, s)
                           : launch_as<__nv_bfloat16, __nv_bfloat16>(a, tiles, s);
    // the next 64 ranks, on top of these (sums of 32-bit values, as within a pass)
    a.z = a.y;
    a.z_stride = a.y_stride;
    a.stall_ns = 0;
  }
  return e;
}

}  // namespace tq
