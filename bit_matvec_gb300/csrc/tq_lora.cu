// tq_lora.cu -- low-rank adapters of many requests beside a shared product:
// Y[t] = Z[t] + scale B (A x[t]) with the adapter of each token.
//
// Tokens of one adapter are taken in tiles of up to 32. A cluster of eight
// thread blocks computes a tile in one launch: each block the products of the
// tile's activations with its eighth of A's columns; the eight partial results
// (32 x rank floats) are summed through distributed shared memory, in the same
// order everywhere; then each block multiplies its share of B's rows and adds Z.
// So A and B are read once a tile, h = A x never leaves the chip, and the only
// traffic that grows with the tokens is x, Z and Y.
//
// Products run on the tensor cores in tf32 (m16n8k8, tokens as rows): f16 and
// bf16 weights are exact in it, a 32-bit activation (and h) is split in two tf32
// parts whose sum is good to 2^-21. The order of the contraction index is free,
// so a thread loads consecutive values of a row and feeds them as the pairs
// (t, t + 4) that the fragment wants.
//
// Tiles are of 8 tokens where there are no more than that for each slot of an adapter on average, used or not: both
// parts of a value are rows of one product then. (Tiles of 32 for 256 tokens of 100 adapters, rank 64, 17408 x
// 5120: 102 us where those of 8 take 69. But 2048 tokens of one adapter in a pool of 256 slots, rank 16, 5120 x 5120,
// take 78 us, and 49 with a description of that slot alone.) Long batches of high rank have a kernel of their own, in
// tq_lora_large.cu. A warp's weights come through a ring of asynchronous copies that only it reads, 6 KB
// under way, so the products wait for no barrier; two thread blocks an SM, 96 KB.
//
// What bounds it: one token, 5120 x 5120, rank 16: 7.1 us of latency (one launch, the token's adapter, A, the
// cluster's sum, B, one after the other). 256 tokens of 100 adapters, ranks 16 to 64: 190 MB in 69 us or
// 2.8 TB/s: some 740 thread blocks of which 304 run at once, each with the same wait for its tile, its first
// weights and the cluster. 8192 tokens of 16 adapters, ranks up to 32, 5120 x 17408: 1.3 GB in 333 us or
// 3.9 TB/s at 1.5 instructions a cycle, conversions and products of the x and Z that pass.
#include <algorithm>

#include "tq_lora.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;        // thread blocks that share a tile
constexpr int kTile = 32;          // tokens of a tile at most: two row blocks of 16
constexpr int kSmallTile = 8;      // or so many, where adapters have few tokens each
constexpr int kParts = 8;          // shares of a block's columns, a warp's each, summed apart
constexpr int kChain = 4;          // chunks of 32 columns that are summed on the tensor cores
constexpr int kInBlock = 256;      // tokens up to which every block finds its tile itself
constexpr int kGroupThreads = 1024;
static_assert(kInBlock == kThreads, "a thread a token");

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- tiles

// The adapter that a token uses, -1 for none, and its rank; `bad` if it is out of range.
__device__ __forceinline__ int effective(const LoraArgs& p, int id, int& rank, bool& bad) {
  bad = false;
  rank = 0;
  if (id < 0) return -1;
  if (id >= p.l.adapters) {
    bad = true;
    return -1;
  }
  rank = p.l.rank ? __ldg(p.l.rank + id) : (int)p.l.max_rank;
  bad = rank < 0 || rank > p.l.max_rank;
  return bad || rank == 0 ? -1 : id;
}

struct Tile {
  int adapter, rank, count;
};

// Up to kInBlock tokens: tile number `want` of the call, its tokens into tok;
// count 0 if there are fewer tiles. Tiles are numbered by their first tokens; a
// token's place among those of its adapter is the number of them before it.
__device__ __forceinline__ Tile find_tile(const LoraArgs& p, int want, bool report, int* tok, int* ids, int* red) {
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  int id = -2, rank = 0;
  bool bad = false;
  if (i < p.ntok) id = effective(p, p.ids[i], rank, bad);
  if (bad && report) atomicMax(p.status, kDevIndex);
  ids[i] = id;
  __syncthreads();
  int before = 0;
  const int whole = warp * 32;   // tokens of the warps before: no comparison of places
  for (int j = 0; j < whole; j += 4) {
    const int4 q = *reinterpret_cast<const int4*>(ids + j);
    before += (q.x == id) + (q.y == id) + (q.z == id) + (q.w == id);
  }
  before += __popc(__match_any_sync(0xffffffffu, id) & ((1u << lane) - 1));
  const bool first = id != -2 && (id >= 0 || p.copy) && before % p.tile == 0;
  const unsigned firsts = __ballot_sync(0xffffffffu, first);
  if (lane == 0) red[warp] = __popc(firsts);
  __syncthreads();
  int number = __popc(firsts & ((1u << lane) - 1));
  for (int w = 0; w < warp; ++w) number += red[w];
  if (first && number == want) {
    red[kWarps] = id;
    red[kWarps + 1] = before;
    red[kWarps + 2] = rank;
    red[kWarps + 3] = 0;
  }
  __syncthreads();
  int total = 0;
  for (int w = 0; w < kWarps; ++w) total += red[w];
  if (want >= total) return {-1, 0, 0};
  const int adapter = red[kWarps], from = red[kWarps + 1];
  const bool mine = id == adapter && before >= from && before < from + p.tile;
  if (mine) tok[before - from] = i;
  const int n = __popc(__ballot_sync(0xffffffffu, mine));
  if (lane == 0 && n) atomicAdd(&red[kWarps + 3], n);
  __syncthreads();
  return {adapter, red[kWarps + 2], red[kWarps + 3]};
}

// More tokens: their order by adapter and the tiles, by one thread block.
// Counters of the adapters (the last one: no adapter) in shared memory. Which of
// an adapter's tokens come first is left to chance: a token's result depends
// neither on its place nor on the other tokens of its tile.
__global__ void __launch_bounds__(kGroupThreads) group_kernel(const __grid_constant__ LoraArgs p, int32_t* order,
                                                              int4* tiles, int* ntiles) {
  extern __shared__ int2 part[];                       // [32], their sum
  int2& total = part[32];
  int* const counts = reinterpret_cast<int*>(part + 33);   // [adapters + 1]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = (int)p.l.adapters + 1;
  for (int g = tid; g < groups; g += kGroupThreads) counts[g] = 0;
  if (tid == 0) total = make_int2(0, 0);
  __syncthreads();
  pdl_wait_primary();
  pdl_launch_dependents();
  auto group_of = [&](int64_t i, bool report) {
    bool bad;
    int rank;
    const int id = effective(p, p.ids[i], rank, bad);
    if (bad && report) atomicMax(p.status, kDevIndex);
    return id < 0 ? (p.copy ? groups - 1 : -1) : id;
  };
  // one addition for all lanes of a group; the place of this lane's token in it
  auto take = [&](int g) {
    const unsigned same = __match_any_sync(0xffffffffu, g);
    const int leader = __ffs(same) - 1;
    int at = 0;
    if (lane == leader && g >= 0) at = atomicAdd(&counts[g], __popc(same));
    return __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1));
  };
  const int64_t whole = ((int64_t)p.ntok + 31) / 32 * 32;
  for (int64_t i = tid; i < whole; i += kGroupThreads) take(i < p.ntok ? group_of(i, true) : -1);
  __syncthreads();
  // where each group's tokens and tiles start
  for (int g0 = 0; g0 < groups; g0 += kGroupThreads) {
    const int g = g0 + tid, n = g < groups ? counts[g] : 0;
    const int tile = g == groups - 1 ? p.copy_tile : p.tile, ntile = n / tile + (n % tile != 0);
    int2 s = make_int2(n, ntile);
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, s.x, d), b = __shfl_up_sync(0xffffffffu, s.y, d);
      if (lane >= d) {
        s.x += a;
        s.y += b;
      }
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    const int2 base = total;
    int2 at = make_int2(base.x + s.x - n, base.y + s.y - ntile);
    int2 sum = make_int2(0, 0);
    for (int w = 0; w < 32; ++w) {
      const int2 q = part[w];
      if (w < warp) {
        at.x += q.x;
        at.y += q.y;
      }
      sum.x += q.x;
      sum.y += q.y;
    }
    __syncthreads();
    if (tid == 0) total = make_int2(base.x + sum.x, base.y + sum.y);
    if (g < groups) {
      counts[g] = at.x;
      const int id = g == groups - 1 ? -1 : g;
      const int rank = id < 0 || n == 0 ? 0 : p.l.rank ? __ldg(p.l.rank + id) : (int)p.l.max_rank;
      for (int k = 0; k < ntile; ++k)
        tiles[at.y + k] = make_int4(id, rank, at.x + k * tile, min(tile, n - k * tile));
    }
    __syncthreads();
  }
  if (tid == 0) *ntiles = total.y;
  for (int64_t i = tid; i < whole; i += kGroupThreads) {
    const int g = i < p.ntok ? group_of(i, false) : -1, at = take(g);
    if (g >= 0) order[at] = (int)i;
  }
}

// ---------------------------------------------------------------- the products

// Asynchronous copies of 16 and 8 bytes into this thread's own slots of shared memory: what a thread
// copies it reads itself, so it waits for nobody. `have`: false gives zeros; `bytes`: zeros behind them.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 slot16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 slot8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void put8(uint32_t a, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
}

// Stages of weights under way, a warp: 6 KB.
__host__ __device__ constexpr int stages(int nt) { return 12 / nt; }
constexpr int kPitch = 33;       // floats of a row of results on their way to rows of Y at any address
// Shared memory in 4-byte words, for adapters of up to `top` rows of A, NT row blocks at a time: the
// tile's description, the partial h of this block's columns, the split h, the warps' stages of weights
// (the first of which also takes the warp's part of h).
constexpr int kHeadInts = kThreads + kTile + 16;
__host__ __device__ constexpr int rank16(int top) { return (top + 15) / 16 * 16; }
__host__ __device__ constexpr int part_floats(int top, bool packed) { return (packed ? 16 : kTile) * rank16(top); }
__host__ __device__ constexpr int split_floats(int top, bool packed) { return (packed ? 16 : 2 * kTile) * rank16(top); }
__host__ __device__ constexpr int stage_floats(int nt) { return nt * 128; }
__host__ __device__ constexpr int ring_floats(int nt) { return kWarps * stages(nt) * stage_floats(nt); }
__host__ __device__ constexpr int pitch_floats(bool packed) { return kWarps * (packed ? 8 : 16) * kPitch; }

// NT: row blocks of 8 of A that a warp takes at a time; ranks above 8 NT take several turns. kPacked:
// small tiles, the two parts of a value as rows g and g + 8 of one product.
template <typename TX, typename TW, int NT, bool kPacked>
__global__ void __launch_bounds__(kThreads, 2)
lora_kernel(const __grid_constant__ LoraArgs p) {
  constexpr bool kSplit = sizeof(TX) == 4;    // 16-bit activations are exact in tf32
  // Chunks of x under way: with one, each chunk waited for the next one's activations. (Small tiles, 256
  // tokens of 100 adapters: 97 us; two 85; three and two thread blocks an SM instead of three 69; six 80.)
  constexpr int kAheadX = kPacked ? 3 : 1;
  constexpr int kBlock = 8 * NT, KG = NT / 2, kStages = stages(NT);
  extern __shared__ float4 shared4[];
  int* const s_ids = reinterpret_cast<int*>(shared4);                // [kThreads]
  int* const s_tok = s_ids + kThreads;                               // [kTile]
  int* const s_red = s_tok + kTile;                                  // [kWarps + 4]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t crank = cluster_rank();
  const int unit = blockIdx.x / kCluster, want = unit / p.splits, part_of = unit % p.splits;
  pdl_wait_primary();
  pdl_launch_dependents();

  Tile tile;
  if (p.tiles) {
    const int n = *p.ntiles;
    const int4 q = p.tiles[want];       // (what is there behind the last one is not used)
    if (want >= n) return;
    tile = {q.x, q.y, q.w};
    if (tid < q.w) s_tok[tid] = p.order[q.z + tid];
    __syncthreads();
  } else {
    tile = find_tile(p, want, blockIdx.x == 0, s_tok, s_ids, s_red);
    if (tile.count == 0) return;
  }
  const int count = tile.count, rank = tile.rank;
  // rows of B and Y of this thread block, in units of 32
  const int rows = (int)p.l.rows, units = (rows + 31) / 32, shares = p.splits * kCluster;
  const int share = part_of * kCluster + (int)crank;
  const int unit0 = (int)((int64_t)units * share / shares), unit1 = (int)((int64_t)units * (share + 1) / shares);

  if (tile.adapter < 0) {   // Z as it is, to the bit
    copy_rows(p, s_tok, count, unit0 * 32, max(0, min(rows, unit1 * 32) - unit0 * 32), kThreads);
    return;
  }
  const float scale = p.l.scale ? __ldg(p.l.scale + tile.adapter) : 1.0f;
  const int wide = rank16(rank);          // values of h a token, with zeros behind the rank
  // Up to 16 tokens: all warps take them; more: half of the warps each 16.
  const int mblocks = !kPacked && count > 16 ? 2 : 1, m = mblocks == 2 ? warp >> 2 : 0;
  const int turn = mblocks == 2 ? warp & 3 : warp, turns = kWarps / mblocks;
  float* const part = reinterpret_cast<float*>(shared4) + kHeadInts; // [kTile][wide]
  uint32_t* const hi = reinterpret_cast<uint32_t*>(part + part_floats((int)p.l.max_rank, kPacked));
  uint32_t* const lo = hi + mblocks * 16 * wide;
  float* const ring = reinterpret_cast<float*>(hi + split_floats((int)p.l.max_rank, kPacked));
  float* const own_ring = ring + warp * kStages * stage_floats(NT);
  const uint32_t slots = smem_u32(own_ring);                          // [kStages][NT][32] pieces of 16 bytes
  float* const pitched = ring + ring_floats(NT) + warp * (kPacked ? 8 : 16) * kPitch;
  const int token[2] = {16 * m + g < count ? s_tok[16 * m + g] : -1,
                        !kPacked && 16 * m + 8 + g < count ? s_tok[16 * m + 8 + g] : -1};

  // ---- h = A x over this block's columns
  const TW* const A = static_cast<const TW*>(p.l.a) + tile.adapter * p.l.a_stride;
  const int cols = (int)p.l.cols, chunks = (cols + 31) / 32;
  const int chunk0 = (int)((int64_t)chunks * crank / kCluster), chunk1 = (int)((int64_t)chunks * (crank + 1) / kCluster);
  const TX* const x0 = static_cast<const TX*>(p.x) + max(token[0], 0) * p.x_stride;
  const TX* const x1 = static_cast<const TX*>(p.x) + max(token[1], 0) * p.x_stride;
  // A share is every eighth chunk of 32 columns; a warp has one, or two with 16 rows for each half of
  // the warps: the sums are the same ones either way.
  for (int r0 = 0; r0 < rank; r0 += kBlock) {
#pragma unroll 1
   for (int share_of = turn; share_of < kParts; share_of += turns) {
    const int mine = max(0, (chunk1 - chunk0 - share_of + kParts - 1) / kParts);     // its chunks
    // The tensor cores cut their sums where 32-bit additions round, which leans
    // one way: every kChain chunks the sum is added to another, by additions that
    // round (without, 2176 columns a warp at rank 256 were 3.3e-6 off, with 2.2e-6).
    float acc[NT][4], sum[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = sum[j][e] = 0.0f;
    // Where this thread's pieces come from: addresses that step from chunk to
    // chunk. Columns past the last are behind every chunk but the last one's.
    constexpr int kStep = kParts * 32;
    const int k0 = (chunk0 + share_of) * 32 + 8 * t;
    const TW* from_a = A + (r0 + g) * p.l.a_row_stride + k0;
    const int64_t block_step = 8 * p.l.a_row_stride;
    const TX* from_x0 = x0 + k0;
    const TX* from_x1 = x1 + k0;
    uint32_t has = 0;               // blocks whose row of this thread there is
#pragma unroll
    for (int j = 0; j < NT; ++j) has |= (r0 + 8 * j + g < rank ? 1u : 0u) << j;
    int ahead = 0, stage_to = 0, stage_from = 0;
    auto issue = [&]() {
      if (ahead < mine) {
        const uint32_t at = slots + stage_to * (stage_floats(NT) * 4) + lane * 16;
        const bool in = k0 + ahead * kStep < cols;    // (cols is a multiple of 8)
        const TW* f = from_a;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const bool have = in && (has >> j & 1u);
          copy16(at + j * 512, have ? f : A, have);
          f += block_step;
        }
        from_a += kStep;
        ++ahead;
        stage_to = stage_to == kStages - 1 ? 0 : stage_to + 1;
      }
      copies_issued();
    };
    auto load_x = [&](int i, Acts<TX> (&v)[2]) {
      const bool in = i < mine && k0 + i * kStep < cols;
      if (in && token[0] >= 0) v[0].load(from_x0);
      else v[0].clear();
      if (!kPacked) {
        if (in && token[1] >= 0) v[1].load(from_x1);
        else v[1].clear();
        from_x1 += kStep;
      }
      from_x0 += kStep;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue();
    Acts<TX> next[kAheadX][2];
#pragma unroll
    for (int i = 0; i < kAheadX; ++i) load_x(i, next[i]);
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      issue();
      Acts<TX> v[2] = {next[0][0], next[0][1]};
#pragma unroll
      for (int u = 0; u + 1 < kAheadX; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) next[u][h] = next[u + 1][h];
      load_x(i + kAheadX, next[kAheadX - 1]);
      copies_but<kStages - 1>();
      uint4 w[NT];
      const uint32_t at = slots + stage_from * (stage_floats(NT) * 4) + lane * 16;
      stage_from = stage_from == kStages - 1 ? 0 : stage_from + 1;
#pragma unroll
      for (int j = 0; j < NT; ++j) w[j] = slot16(at + j * 512);
      __syncwarp();     // the products take a whole warp
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t fa[4], fb[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a = 0, b = 0;
          if (!kPacked || h == 0) v[h].pair(s, a, b);
          if constexpr (kSplit) {
            split(__uint_as_float(a), fa[h], fb[h]);
            split(__uint_as_float(b), fa[2 + h], fb[2 + h]);
          } else {
            fa[h] = a;
            fa[2 + h] = b;
          }
        }
        if (kSplit && kPacked) {
          fa[1] = fb[0];
          fa[3] = fb[2];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (r0 + 8 * j >= rank) break;
          uint32_t b0, b1;
          widen<TW>(s == 0 ? w[j].x : s == 1 ? w[j].y : s == 2 ? w[j].z : w[j].w, b0, b1);
          mma_tf32(acc[j], fa, b0, b1);
          if (kSplit && !kPacked) mma_tf32(acc[j], fb, b0, b1);
        }
      }
      if (i % kChain == kChain - 1 || i == mine - 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum[j][e] += acc[j][e];
            acc[j][e] = 0.0f;
          }
      }
    }
    // to where the shares are summed: a warp's last one in its first stage
    copies_but<0>();
    float* const place = share_of + turns < kParts ? pitched : own_ring;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float* const to = place + g * kBlock + 8 * j + 2 * t;
      if (kPacked) {
        // (16-bit activations have no second part: its sums are zeros, or NaN of infinite weights)
        *reinterpret_cast<float2*>(to) = kSplit ? make_float2(sum[j][0] + sum[j][2], sum[j][1] + sum[j][3])
                                                : make_float2(sum[j][0], sum[j][1]);
        *reinterpret_cast<float2*>(to + 8 * kBlock) = make_float2(0.0f, 0.0f);
      } else {
        *reinterpret_cast<float2*>(to) = make_float2(sum[j][0], sum[j][1]);
        *reinterpret_cast<float2*>(to + 8 * kBlock) = make_float2(sum[j][2], sum[j][3]);
      }
    }
   }
    __syncthreads();
    const int here = min(kBlock, wide - r0);
    for (int i = tid; i < mblocks * 16 * kBlock; i += kThreads) {
      const int j = i / kBlock, r = i % kBlock, first = (j >> 4) * turns, at = (j & 15) * kBlock + r;
      if (r >= here) continue;
      float total = 0.0f;
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        const int w = first + (q & (turns - 1));
        total += (q + turns < kParts ? ring + ring_floats(NT) + w * 16 * kPitch : ring + w * kStages * stage_floats(NT))[at];
      }
      part[j * wide + r0 + r] = total;
    }
    __syncthreads();
  }

  // ---- Y = Z + B h: what it starts with is on its way while the blocks wait for one another
  const TW* const B = static_cast<const TW*>(p.l.b) + tile.adapter * p.l.b_stride;
  const int groups = wide / 16, turns_b = (groups + KG - 1) / KG;      // turns of 16 KG values of h a unit
  const int items = max(0, (unit1 - unit0 - turn + turns - 1) / turns) * turns_b;
  // Column g of block i is row 8 (g / 2) + 2 i + g % 2, so that a thread's results are consecutive rows.
  const int row_of = 8 * (g >> 1) + (g & 1);
  int unit_ahead = unit0 + turn, turn_ahead = 0, ahead = 0, stage_to = 0, stage_from = 0;
  const int64_t pair_step = 2 * p.l.b_row_stride;
  const TW* from_b = B + (unit_ahead * 32 + row_of) * p.l.b_row_stride + 4 * t;   // of the unit ahead
  const bool whole_b = p.b_vec && rank % 4 == 0;     // a thread's four values all there, or none
  auto issue = [&]() {
    if (ahead < items) {
      const uint32_t at = slots + stage_to * (stage_floats(NT) * 4) + lane * 8;
      const int k0 = 16 * KG * turn_ahead;
      if (whole_b && unit_ahead * 32 + 32 <= rows) {
        const TW* f = from_b + k0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int q = 0; q < KG; ++q) {
            const bool have = k0 + 16 * q + 4 * t < rank;
            copy8(at + (q * 4 + i) * 256, have ? f + 16 * q : B, have ? 8 : 0);
          }
          f += pair_step;
        }
      } else if (p.b_pairs) {
        const TW* f = from_b + k0;
        const int rows_left = rows - unit_ahead * 32 - row_of, left = rank - k0 - 4 * t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int q = 0; q < KG; ++q) {
            const int have = 2 * i < rows_left ? min(8, max(0, 2 * left - 32 * q)) : 0;
            const uint32_t to = at + (q * 4 + i) * 256;
            const TW* const from = have ? f + 16 * q : B;
            if (p.b_vec) {
              copy8(to, from, have);
            } else {
              copy4(to, from, min(have, 4));
              copy4(to + 4, have > 4 ? from + 2 : B, max(have - 4, 0));
            }
          }
          f += pair_step;
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < KG; ++q) {
          const int k = k0 + 16 * q + 4 * t;
          uint32_t v[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int n = unit_ahead * 32 + row_of + 2 * i;
              v[i][e] = n < rows && k + e < rank
                            ? __ldg(reinterpret_cast<const unsigned short*>(B + n * p.l.b_row_stride + k) + e) : 0u;
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            put8(at + (q * 4 + i) * 256, make_uint2(v[i][0] | v[i][1] << 16, v[i][2] | v[i][3] << 16));
        }
      }
      if (++turn_ahead == turns_b) {
        turn_ahead = 0;
        unit_ahead += turns;
        from_b += 32 * turns * p.l.b_row_stride;
      }
      ++ahead;
      stage_to = stage_to == kStages - 1 ? 0 : stage_to + 1;
    }
    copies_issued();
  };
  const bool vec = p.y_vec && p.z_vec;
  const int bytes = p.y_type == TQ_F32 ? 4 : 2;
  const char* from_z[2];
  char* to_y[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = (unit0 + turn) * 32 + 8 * t, j = max(token[h], 0);
    from_z[h] = static_cast<const char*>(p.z) + (j * p.z_stride + at) * bytes;
    to_y[h] = static_cast<char*>(p.y) + (j * p.y_stride + at) * bytes;
  }
  // Z of 16 tokens and 32 rows: the eight rows of this thread's two tokens, or
  // (rows of Y or Z at any address, or the last of them) a row of each of the 16
  auto load_z = [&](int u, uint32_t (&z)[16]) {
    if (p.z && u < unit1) {
      const int n0 = u * 32;
      if (vec && n0 + 32 <= rows) {
#pragma unroll
        for (int h = 0; h < (kPacked ? 1 : 2); ++h)
          if (token[h] >= 0) load8(from_z[h], p.y_type, 0, z + 8 * h);
      } else {
        const int have = n0 + lane < rows ? count - 16 * m : 0;
#pragma unroll
        for (int j0 = 0; j0 < (kPacked ? 8 : 16); j0 += 4) {
          const int4 q = *reinterpret_cast<const int4*>(s_tok + 16 * m + j0);
          const int tok[4] = {q.x, q.y, q.z, q.w};
          if (p.y_type == TQ_F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j0 + e < have) z[j0 + e] = (static_cast<const uint32_t*>(p.z) + n0 + lane)[tok[e] * p.z_stride];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j0 + e < have) z[j0 + e] = (static_cast<const uint16_t*>(p.z) + n0 + lane)[tok[e] * p.z_stride];
          }
        }
      }
    }
    from_z[0] += 32 * turns * bytes;
    if (!kPacked) from_z[1] += 32 * turns * bytes;
  };
  uint32_t z_next[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) z_next[e] = 0;
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) issue();
  load_z(unit0 + turn, z_next);
  cluster_arrive();
  cluster_wait();

  // ---- h of all columns, split, in the order of the fragments: for each 8 values
  // of h and 16 tokens, a lane's four values
  {
    const uint32_t base = smem_u32(part);
    const int quads = wide / 4, tokens = kPacked ? 8 : mblocks * 16;
    for (int i = tid; i < tokens * quads; i += kThreads) {
      const int j = i / quads, q = i % quads;     // values 4 q .. 4 q + 3 of token j
      float4 v[kCluster];
#pragma unroll
      for (int c = 0; c < kCluster; ++c) v[c] = load_remote(base + (j * wide + 4 * q) * 4, c);
      float h[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        h[0] += v[c].x;
        h[1] += v[c].y;
        h[2] += v[c].z;
        h[3] += v[c].w;
      }
      const int mb = j >> 4, half = (j >> 3) & 1, l = (j & 7) * 4 + (q & 3);
      const float sum = (h[0] + h[1]) + (h[2] + h[3]);      // (NaN if one of them is)
      if (kSplit && sum != sum && j < count) {
        const float4 again = dots_again(make_float4(h[0], h[1], h[2], h[3]), static_cast<const TX*>(p.x) + s_tok[j] * p.x_stride,
                                        A, p.l.a_row_stride, 4 * q, rank, cols);
        h[0] = again.x;
        h[1] = again.y;
        h[2] = again.z;
        h[3] = again.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int step = 2 * (q >> 2) + (e >> 1);
        const int at = ((step * mblocks + mb) * 32 + l) * 4 + half + 2 * (e & 1);
        // (past the rank an infinite activation has left a NaN)
        uint32_t a, b;
        split(4 * q + e < rank ? h[e] * scale : 0.0f, a, b);
        hi[at] = a;
        (kPacked ? hi + 1 : lo)[at] = b;
      }
    }
  }
  __syncthreads();
  cluster_arrive();     // this block's part has no reader left when all have arrived

#pragma unroll 1
  for (int u = unit0 + turn; u < unit1; u += turns) {
    const int n0 = u * 32;
    uint32_t z[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = z_next[e];
    load_z(u + turns, z_next);
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
#pragma unroll 1
    for (int q0 = 0; q0 < groups; q0 += KG) {
      issue();
      copies_but<kStages - 1>();
      const uint32_t from = slots + stage_from * (stage_floats(NT) * 4) + lane * 8;
      stage_from = stage_from == kStages - 1 ? 0 : stage_from + 1;
      uint2 w[KG][4];
#pragma unroll
      for (int q = 0; q < KG; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[q][i] = slot8(from + (q * 4 + i) * 256);
      __syncwarp();
#pragma unroll
      for (int q = 0; q < KG; ++q) {
        if (q0 + q >= groups) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int at = (((2 * (q0 + q) + s) * mblocks + m) * 32 + lane) * 4;
          const uint4 a = *reinterpret_cast<const uint4*>(hi + at);
          const uint32_t fa[4] = {a.x, a.y, a.z, a.w};
          uint4 b = make_uint4(0, 0, 0, 0);
          if (!kPacked) b = *reinterpret_cast<const uint4*>(lo + at);
          const uint32_t fb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            widen<TW>(s ? w[q][i].y : w[q][i].x, b0, b1);
            mma_tf32(acc[i], fa, b0, b1);
            if (!kPacked) mma_tf32(acc[i], fb, b0, b1);
          }
        }
      }
    }
    if (kPacked) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][0] = joined(acc[i][0], acc[i][2]);
        acc[i][1] = joined(acc[i][1], acc[i][3]);
      }
    } else {
      // A NaN among this thread's sums (or infinities of both signs) is one in their sum.
      uint64_t some[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) some[h] = tc::f2_add(some[h], tc::f2_packf(acc[i][2 * h], acc[i][2 * h + 1]));
      const float2 two = tc::f2_unpack(tc::f2_add(some[0], some[1]));
      const float all = two.x + two.y;
      if (__any_sync(0xffffffffu, all != all)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e) pitched[(8 * h + g) * kPitch + 8 * t + e] = acc[e >> 1][2 * h + (e & 1)];
        __syncwarp();
        // a row of B a lane, one token after the other
#pragma unroll 1
        for (int j = 16 * m; n0 + lane < rows && j < min(count, 16 * m + 16); ++j) {
          float& y = pitched[(j - 16 * m) * kPitch + lane];
          if (y == y) continue;
          y = row_again(reinterpret_cast<const float*>(hi), reinterpret_cast<const float*>(lo), [&](int r) {
            const int step = 2 * (r >> 4) + ((r >> 1) & 1), l = (j & 7) * 4 + ((r >> 2) & 3);
            return ((step * mblocks + (j >> 4)) * 32 + l) * 4 + ((j >> 3) & 1) + 2 * (r & 1);
          }, B + (n0 + lane) * p.l.b_row_stride, rank);
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e >> 1][2 * h + (e & 1)] = pitched[(8 * h + g) * kPitch + 8 * t + e];
        __syncwarp();
      }
    }
    if (vec && n0 + 32 <= rows) {
#pragma unroll
      for (int h = 0; h < (kPacked ? 1 : 2); ++h) {
        if (token[h] < 0) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = p.y_type == TQ_F32 ? __uint_as_float(z[8 * h + e])
                                    : up((uint16_t)(z[8 * h + (e >> 1)] >> (16 * (e & 1))), p.y_type);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += acc[e >> 1][2 * h + (e & 1)];
        store8(to_y[h], p.y_type, 0, v);
      }
    } else {
      // rows of Y at any address: through shared memory, so that a warp stores
      // 32 rows of a token
#pragma unroll
      for (int h = 0; h < (kPacked ? 1 : 2); ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) pitched[(8 * h + g) * kPitch + 8 * t + e] = acc[e >> 1][2 * h + (e & 1)];
      __syncwarp();
      // (four tokens at a time, no branch between them: 170 cycles each otherwise)
      const int have = n0 + lane < rows ? count - 16 * m : 0;
#pragma unroll
      for (int j0 = 0; j0 < (kPacked ? 8 : 16); j0 += 4) {
        const int4 q = *reinterpret_cast<const int4*>(s_tok + 16 * m + j0);
        const int tok[4] = {q.x, q.y, q.z, q.w};
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = up1(z[j0 + e], p.y_type) + pitched[(j0 + e) * kPitch + lane];
        if (p.y_type == TQ_F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j0 + e < have) (static_cast<float*>(p.y) + n0 + lane)[tok[e] * p.y_stride] = v[e];
        } else {
          uint16_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = down(v[e], p.y_type);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j0 + e < have) (static_cast<uint16_t*>(p.y) + n0 + lane)[tok[e] * p.y_stride] = w[e];
        }
      }
      __syncwarp();
    }
    to_y[0] += 32 * turns * bytes;
    if (!kPacked) to_y[1] += 32 * turns * bytes;
  }
  copies_but<0>();
  cluster_wait();
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Tiles of 8 tokens where slots have no more than that each on average. (A function of the call's
// sizes alone: so is the order of every sum.)
int64_t tile_of(int64_t ntok, int64_t adapters) { return ntok <= kSmallTile * adapters ? kSmallTile : kTile; }
int64_t max_tiles(int64_t ntok, int64_t adapters, int64_t tile) {
  return std::min(ntok, ntok / tile + std::min(adapters, ntok) + 1);
}

bool in_pieces(const void* p, int64_t stride, int64_t bytes, int64_t piece) {
  return (uintptr_t)p % piece == 0 && stride * bytes % piece == 0;
}

template <typename TX, typename TW, int NT, bool kPacked>
cudaError_t launch_as(const LoraArgs& a, int64_t tiles, cudaStream_t s) {
  const auto kernel = lora_kernel<TX, TW, NT, kPacked>;
  const int top = (int)a.l.max_rank;
  const int smem = (kHeadInts + part_floats(top, kPacked) + split_floats(top, kPacked) + ring_floats(NT) + pitch_floats(kPacked)) * (int)sizeof(float);
  cudaError_t e = ensure_dynamic_smem((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t grid = tiles * a.splits * kCluster;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
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

template <typename TX, typename TW>
cudaError_t launch_for(const LoraArgs& a, int64_t tiles, cudaStream_t s) {
  if (a.tile == kSmallTile)
    return a.l.max_rank <= 16 ? launch_as<TX, TW, 2, true>(a, tiles, s) : launch_as<TX, TW, 4, true>(a, tiles, s);
  return a.l.max_rank <= 16 ? launch_as<TX, TW, 2, false>(a, tiles, s) : launch_as<TX, TW, 4, false>(a, tiles, s);
}

}  // namespace

// The order of the tokens, the tiles and their number.
int64_t lora_workspace_bytes(int64_t ntok, int64_t adapters) {
  if (ntok <= kInBlock) return 0;
  return 16 + max_tiles(ntok, adapters, tile_of(ntok, adapters)) * 16 + ceil_div(ntok, 4) * 16;
}

cudaError_t launch_lora_add(const LoraCall& c, cudaStream_t s) {
  LoraArgs a = {};
  a.x = c.x;
  a.z = c.z;
  a.y = c.y;
  a.ids = c.ids;
  a.l = c.lora;
  a.x_stride = c.x_stride;
  a.z_stride = c.z_stride;
  a.y_stride = c.y_stride;
  a.y_type = c.y_type;
  a.ntok = (int)c.ntok;
  a.copy = c.z != c.y;
  a.status = c.status;
  const int64_t yb = c.y_type == TQ_F32 ? 4 : 2;
  a.y_vec = in_pieces(c.y, c.ntok > 1 ? c.y_stride : 0, yb, 16);
  a.z_vec = in_pieces(c.z, c.ntok > 1 ? c.z_stride : 0, yb, 16);
  a.b_vec = in_pieces(c.lora.b, c.lora.rows > 1 ? c.lora.b_row_stride : 0, 2, 8) &&
            in_pieces(nullptr, c.lora.adapters > 1 ? c.lora.b_stride : 0, 2, 8);
  a.b_pairs = in_pieces(c.lora.b, c.lora.rows > 1 ? c.lora.b_row_stride : 0, 2, 4) &&
              in_pieces(nullptr, c.lora.adapters > 1 ? c.lora.b_stride : 0, 2, 4);
  const bool large = lora_large_fits(a, c.ntok);
  a.tile = large ? kLargeTile : (int)tile_of(c.ntok, c.lora.adapters);
  // (tokens without adapter are copied, 32 to a tile, which is quick)
  a.copy_tile = (int)std::min<int64_t>(a.tile, kTile);
  const int64_t tiles = max_tiles(c.ntok, c.lora.adapters, a.copy ? a.copy_tile : a.tile);
  // Few tiles: several clusters share the rows of one, each with the whole of h
  // for itself, up to as many thread blocks as run at once, and while a block's share of B and
  // Y is no less than half its share of A and x.
  const int64_t r = std::max<int64_t>(c.lora.max_rank, 1);
  const int64_t most = std::max<int64_t>(1, 2 * c.lora.rows * (r + 4) / std::max<int64_t>(1, c.lora.cols * (r + 2)));
  a.splits = (int)std::max<int64_t>(1, std::min(most, 304 / (tiles * kCluster)));
  if (c.ntok > kInBlock) {
    char* at = static_cast<char*>(c.ws);
    int* ntiles = reinterpret_cast<int*>(at);
    int4* list = reinterpret_cast<int4*>(at + 16);
    int32_t* order = reinterpret_cast<int32_t*>(at + 16 + tiles * 16);
    const int smem = (int)(c.lora.adapters + 1) * 4 + 33 * 8;
    cudaError_t e = ensure_dynamic_smem((const void*)group_kernel, smem);
    if (e == cudaSuccess)
      e = launch_pdl(group_kernel, dim3(1), dim3(kGroupThreads), (size_t)smem, s, a, order, list, ntiles);
    if (e != cudaSuccess) return e;
    a.order = order;
    a.tiles = list;
    a.ntiles = ntiles;
  }
  if (large) return launch_lora_large(a, tiles, c.x_type, s);
  if (c.lora.type == TQ_F16)
    return c.x_type == TQ_F32 ? launch_for<float, __half>(a, tiles, s) : launch_for<__half, __half>(a, tiles, s);
  return c.x_type == TQ_F32 ? launch_for<float, __nv_bfloat16>(a, tiles, s)
                            : launch_for<__nv_bfloat16, __nv_bfloat16>(a, tiles, s);
}

}  // namespace tq
