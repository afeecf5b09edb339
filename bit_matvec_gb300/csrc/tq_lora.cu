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
#include <algorithm>

#include "tq_requests.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kTile = 32;          // tokens of a tile: two row blocks of 16
constexpr int kChain = 4;          // chunks of 32 columns that are summed on the tensor cores
constexpr int kInBlock = 256;      // tokens up to which every block finds its tile itself
constexpr int kGroupThreads = 1024;
static_assert(kInBlock == kThreads, "a thread a token");

struct Args {
  const void* x;
  const void* z;
  void* y;
  const int32_t* ids;
  tq_lora l;
  int64_t x_stride, z_stride, y_stride;
  int y_type;
  int ntok;
  int splits;            // clusters that share the rows of a tile
  int copy;              // tokens without adapter are copied (Z is not Y)
  int y_vec, z_vec;      // rows of Y, of Z in 16-byte pieces
  int b_vec;             // rows of B in 8-byte pieces
  // more than kInBlock tokens: the tiles, from the grouping kernel
  const int32_t* order;  // tokens by adapter
  const int4* tiles;     // adapter, its rank, first of order, tokens
  const int* ntiles;
  int* status;
};

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x as a tf32 value and the rest of it, rounded to tf32: good to 2^-21. The
// first part is cut, not rounded, so that it does not overflow; an infinity
// leaves no rest.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  const float h = __uint_as_float(hi), rest = x == h ? 0.0f : x - h;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
}

// The two 16-bit values of a word as 32-bit ones.
template <typename T> __device__ __forceinline__ void widen(uint32_t w, uint32_t& a, uint32_t& b);
template <> __device__ __forceinline__ void widen<__nv_bfloat16>(uint32_t w, uint32_t& a, uint32_t& b) {
  a = w << 16;
  b = w & 0xffff0000u;
}
template <> __device__ __forceinline__ void widen<__half>(uint32_t w, uint32_t& a, uint32_t& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = __float_as_uint(f.x);
  b = __float_as_uint(f.y);
}

// Eight activations from p on: 32 or 16 bytes.
template <typename TX> struct Acts {
  uint4 v[sizeof(TX) == 4 ? 2 : 1];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (auto& q : v) q = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const TX* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(v) / sizeof(v[0])); ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  // values 2 s and 2 s + 1
  __device__ __forceinline__ void pair(int s, uint32_t& a, uint32_t& b) const {
    if constexpr (sizeof(TX) == 4) {
      const uint4 q = v[s >> 1];
      a = s & 1 ? q.z : q.x;
      b = s & 1 ? q.w : q.y;
    } else {
      const uint4 q = v[0];
      widen<TX>(s == 0 ? q.x : s == 1 ? q.y : s == 2 ? q.z : q.w, a, b);
    }
  }
};

// ---------------------------------------------------------------- Y and Z

__device__ __forceinline__ float up(uint16_t v, int type) {
  return type == TQ_F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ uint16_t down(float v, int type) {
  return type == TQ_F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// n of eight consecutive values from `at` on, as they are (vec: the address is a multiple of 16
// bytes), and as floats.
struct Raw8 {
  uint4 v[2];
};
__device__ __forceinline__ Raw8 load8(const void* p, int type, int64_t at, int n, bool vec) {
  Raw8 r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (type == TQ_F32) {
    const uint32_t* f = static_cast<const uint32_t*>(p) + at;
    if (vec && n == 8) {
      r.v[0] = *reinterpret_cast<const uint4*>(f);
      r.v[1] = *reinterpret_cast<const uint4*>(f + 4);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = e < n ? f[e] : 0u;
      r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
      r.v[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return r;
  }
  const uint16_t* h = static_cast<const uint16_t*>(p) + at;
  if (vec && n == 8) {
    r.v[0] = *reinterpret_cast<const uint4*>(h);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = e < n ? h[e] : 0u;
    r.v[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  return r;
}
__device__ __forceinline__ void floats8(const Raw8& r, int type, float (&v)[8]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
  if (type == TQ_F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = up((uint16_t)(w[e >> 1] >> (16 * (e & 1))), type);
  }
}
__device__ __forceinline__ void store8(void* p, int type, int64_t at, int n, bool vec, const float (&v)[8]) {
  if (type == TQ_F32) {
    float* f = static_cast<float*>(p) + at;
    if (vec && n == 8) {
      *reinterpret_cast<float4*>(f) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(f + 4) = make_float4(v[4], v[5], v[6], v[7]);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) f[e] = v[e];
    return;
  }
  uint16_t* h = static_cast<uint16_t*>(p) + at;
  uint16_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = down(v[e], type);
  if (vec && n == 8) {
    *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(w);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) h[e] = w[e];
}

// ---------------------------------------------------------------- tiles

// The adapter that a token uses, -1 for none, and its rank; `bad` if it is out of range.
__device__ __forceinline__ int effective(const Args& p, int id, int& rank, bool& bad) {
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
__device__ __forceinline__ Tile find_tile(const Args& p, int want, bool report, int* tok, int* ids, int* red) {
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
  const bool first = id != -2 && (id >= 0 || p.copy) && before % kTile == 0;
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
  const bool mine = id == adapter && before >= from && before < from + kTile;
  if (mine) tok[before - from] = i;
  const int n = __popc(__ballot_sync(0xffffffffu, mine));
  if (lane == 0 && n) atomicAdd(&red[kWarps + 3], n);
  __syncthreads();
  return {adapter, red[kWarps + 2], red[kWarps + 3]};
}

// More tokens: their order by adapter and the tiles, by one thread block.
// Counters of the adapters (the last one: no adapter) in shared memory. Which of
// an adapter's tokens come first is left to chance: a token's result does not
// depend on its place.
__global__ void __launch_bounds__(kGroupThreads) group_kernel(const __grid_constant__ Args p, int32_t* order,
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
  auto group_of = [&](int i, bool report) {
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
  const int whole = (p.ntok + 31) & ~31;
  for (int i = tid; i < whole; i += kGroupThreads) take(i < p.ntok ? group_of(i, true) : -1);
  __syncthreads();
  // where each group's tokens and tiles start
  for (int g0 = 0; g0 < groups; g0 += kGroupThreads) {
    const int g = g0 + tid, n = g < groups ? counts[g] : 0;
    int2 s = make_int2(n, (n + kTile - 1) / kTile);
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
    int2 at = make_int2(base.x + s.x - n, base.y + s.y - (n + kTile - 1) / kTile);
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
      for (int k = 0; k * kTile < n; ++k)
        tiles[at.y + k] = make_int4(id, rank, at.x + k * kTile, min(kTile, n - k * kTile));
    }
    __syncthreads();
  }
  if (tid == 0) *ntiles = total.y;
  for (int i = tid; i < whole; i += kGroupThreads) {
    const int g = i < p.ntok ? group_of(i, false) : -1, at = take(g);
    if (g >= 0) order[at] = i;
  }
}

// ---------------------------------------------------------------- the products

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 load_remote(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// Shared memory in 4-byte words, for adapters of up to `top` rows of A in blocks of `block`: the
// tile's description, the partial h of this block's columns, and the eight warps' parts of it, whose
// place the split h takes afterwards.
constexpr int kHeadInts = kThreads + kTile + 16;
__host__ __device__ constexpr int rank16(int top) { return (top + 15) / 16 * 16; }
__host__ __device__ constexpr int part_floats(int top) { return kTile * rank16(top); }
__host__ __device__ constexpr int work_floats(int top, int block) {
  const int warps = kWarps * 16 * block, h = 2 * kTile * rank16(top);
  return warps > h ? warps : h;
}

// What a warp needs of 32 rows of B and Y for 16 tokens, beside h: a thread's values of B for up to
// 16 KG values of h, and of Z for its two tokens and eight rows.
template <typename TW, int KG> struct Unit {
  uint2 w[KG][4];
  Raw8 z[2];
  int64_t out;    // the first of its eight rows of Y
  int some;       // how many of them there are

  // Column g of block i is row 8 (g / 2) + 2 i + g % 2, so that a thread's results are consecutive rows.
  __device__ __forceinline__ void load_b(const Args& p, const TW* B, int64_t n0, int k0, int rank, int g, int t) {
#pragma unroll
    for (int q = 0; q < KG; ++q) {
      const int k = k0 + 16 * q + 4 * t;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + 8 * (g >> 1) + 2 * i + (g & 1);
        const TW* const b = B + n * p.l.b_row_stride + k;
        w[q][i] = make_uint2(0, 0);
        if (p.b_vec && k + 4 <= rank && n < p.l.rows) {
          w[q][i] = __ldg(reinterpret_cast<const uint2*>(b));
        } else if (n < p.l.rows && k < rank) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = k + e < rank ? __ldg(reinterpret_cast<const unsigned short*>(b) + e) : 0u;
          w[q][i] = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
        }
      }
    }
  }
  __device__ __forceinline__ void load_z(const Args& p, int64_t n0, const int (&token)[2], int t) {
    out = n0 + 8 * t;
    some = (int)max((int64_t)0, min((int64_t)8, p.l.rows - out));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (p.z && token[h] >= 0 && some > 0) {
        z[h] = load8(p.z, p.y_type, token[h] * p.z_stride + out, some, p.z_vec);
      } else {
        z[h].v[0] = z[h].v[1] = make_uint4(0, 0, 0, 0);
      }
    }
  }
};

// NT: row blocks of 8 of A that a warp takes at a time; ranks above 8 NT take several turns.
template <typename TX, typename TW, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 4 ? 3 : 2)
lora_kernel(const __grid_constant__ Args p) {
  constexpr bool kSplit = sizeof(TX) == 4;    // 16-bit activations are exact in tf32
  constexpr int kBlock = 8 * NT, KG = NT / 2;
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
    if (want >= *p.ntiles) return;
    const int4 q = p.tiles[want];
    tile = {q.x, q.y, q.w};
    if (tid < q.w) s_tok[tid] = p.order[q.z + tid];
    __syncthreads();
  } else {
    tile = find_tile(p, want, blockIdx.x == 0, s_tok, s_ids, s_red);
    if (tile.count == 0) return;
  }
  const int count = tile.count, rank = tile.rank;
  // rows of B and Y of this thread block, in units of 32
  const int64_t rows = p.l.rows, units = (rows + 31) / 32, shares = (int64_t)p.splits * kCluster;
  const int64_t share = (int64_t)part_of * kCluster + crank;
  const int64_t unit0 = units * share / shares, unit1 = units * (share + 1) / shares;

  if (tile.adapter < 0) {   // Z as it is, to the bit
    for (int j = 0; j < count; ++j) {
      const int64_t to = s_tok[j] * p.y_stride, from = s_tok[j] * p.z_stride;
      const int64_t end = min(rows, unit1 * 32);
      if (p.y_type == TQ_F32) {
        for (int64_t n = unit0 * 32 + tid; n < end; n += kThreads)
          static_cast<uint32_t*>(p.y)[to + n] = p.z ? static_cast<const uint32_t*>(p.z)[from + n] : 0u;
      } else {
        for (int64_t n = unit0 * 32 + tid; n < end; n += kThreads)
          static_cast<uint16_t*>(p.y)[to + n] = p.z ? static_cast<const uint16_t*>(p.z)[from + n] : (uint16_t)0;
      }
    }
    return;
  }
  const float scale = p.l.scale ? __ldg(p.l.scale + tile.adapter) : 1.0f;
  const int wide = rank16(rank);          // values of h a token, with zeros behind the rank
  // up to 16 tokens: all warps take them; more: half of the warps each 16
  const int mblocks = count > 16 ? 2 : 1, m = mblocks == 2 ? warp >> 2 : 0;
  const int turn = mblocks == 2 ? warp & 3 : warp, turns = kWarps / mblocks;
  float* const part = reinterpret_cast<float*>(shared4) + kHeadInts; // [kTile][wide]
  float* const work = part + part_floats((int)p.l.max_rank);         // [kWarps][16][kBlock], then h
  const int token[2] = {16 * m + g < count ? s_tok[16 * m + g] : -1,
                        16 * m + 8 + g < count ? s_tok[16 * m + 8 + g] : -1};

  // ---- h = A x over this block's columns
  const TW* const A = static_cast<const TW*>(p.l.a) + tile.adapter * p.l.a_stride;
  const int cols = (int)p.l.cols, chunks = (cols + 31) / 32;
  const int chunk0 = (int)((int64_t)chunks * crank / kCluster), chunk1 = (int)((int64_t)chunks * (crank + 1) / kCluster);
  const TX* const x0 = static_cast<const TX*>(p.x) + token[0] * p.x_stride;
  const TX* const x1 = static_cast<const TX*>(p.x) + token[1] * p.x_stride;
  for (int r0 = 0; r0 < rank; r0 += kBlock) {
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    const TW* const Ar = A + (r0 + g) * p.l.a_row_stride;
    if (r0 > 0) __syncthreads();
    // The tensor cores cut their sums where 32-bit additions round, which leans
    // one way: after a few chunks the sum goes to this thread's place in shared
    // memory, by an addition that rounds (256 of 2176 columns a warp's chain
    // long, rank 256: 2.2e-6 of the result; without, 3.3e-6).
    float* const mine = work + (warp * 16 + g) * kBlock + 2 * t;
    auto flush = [&](bool first) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2* const at = reinterpret_cast<float2*>(mine + 8 * h * kBlock + 8 * j);
          float2 sum = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
          if (!first) {
            const float2 old = *at;
            sum.x += old.x;
            sum.y += old.y;
          }
          *at = sum;
          acc[j][2 * h] = acc[j][2 * h + 1] = 0.0f;
        }
    };
    int done = 0;
#pragma unroll 2
    for (int c = chunk0 + turn; c < chunk1; c += turns, ++done) {
      if (done > 0 && done % kChain == 0) flush(done == kChain);
      const int k = c * 32 + 8 * t;
      const bool in = k < cols;       // (cols is a multiple of 8)
      uint4 w[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        w[j] = in && r0 + 8 * j + g < rank
                   ? __ldg(reinterpret_cast<const uint4*>(Ar + 8 * j * p.l.a_row_stride + k))
                   : make_uint4(0, 0, 0, 0);
      Acts<TX> v[2];
      if (in && token[0] >= 0) v[0].load(x0 + k);
      else v[0].clear();
      if (in && token[1] >= 0) v[1].load(x1 + k);
      else v[1].clear();
      __syncwarp();     // the products take a whole warp
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a, b;
          v[h].pair(s, a, b);
          if constexpr (kSplit) {
            split(__uint_as_float(a), hi[h], lo[h]);
            split(__uint_as_float(b), hi[2 + h], lo[2 + h]);
          } else {
            hi[h] = a;
            hi[2 + h] = b;
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (r0 + 8 * j >= rank) break;
          uint32_t b0, b1;
          widen<TW>(s == 0 ? w[j].x : s == 1 ? w[j].y : s == 2 ? w[j].z : w[j].w, b0, b1);
          mma_tf32(acc[j], hi, b0, b1);
          if constexpr (kSplit) mma_tf32(acc[j], lo, b0, b1);
        }
      }
    }
    // the warps' parts, summed in their order
    flush(done <= kChain);
    __syncthreads();
    const int here = min(kBlock, wide - r0);
    for (int i = tid; i < mblocks * 16 * kBlock; i += kThreads) {
      const int j = i / kBlock, r = i % kBlock;
      if (r >= here) continue;
      const int first = (j >> 4) * turns;
      float sum = 0.0f;
      for (int w = 0; w < turns; ++w) sum += work[((first + w) * 16 + (j & 15)) * kBlock + r];
      part[j * wide + r0 + r] = sum;
    }
  }
  // what the second product starts with is on its way while the blocks wait for one another
  const TW* const B = static_cast<const TW*>(p.l.b) + tile.adapter * p.l.b_stride;
  Unit<TW, KG> in;
  if (unit0 + turn < unit1) {
    in.load_z(p, (unit0 + turn) * 32, token, t);
    in.load_b(p, B, (unit0 + turn) * 32, 0, rank, g, t);
  }
  cluster_arrive();
  cluster_wait();

  // ---- h of all columns, split, in the order of the fragments: for each 8 values
  // of h and 16 tokens, a lane's four values
  uint32_t* const hi = reinterpret_cast<uint32_t*>(work);
  uint32_t* const lo = hi + mblocks * 16 * wide;
  {
    const uint32_t base = smem_u32(part);
    for (int i = tid; i < mblocks * 16 * wide / 4; i += kThreads) {
      const int j = i / (wide / 4), q = i % (wide / 4);     // values 4 q .. 4 q + 3 of token j
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
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int step = 2 * (q >> 2) + (e >> 1);
        const int at = ((step * mblocks + mb) * 32 + l) * 4 + half + 2 * (e & 1);
        // (past the rank an infinite activation has left a NaN)
        split(4 * q + e < rank ? h[e] * scale : 0.0f, hi[at], lo[at]);
      }
    }
  }
  __syncthreads();
  cluster_arrive();     // this block's part has no reader left when all have arrived

  // ---- Y = Z + B h
  const int groups = wide / 16;
  bool loaded = true;
#pragma unroll 1
  for (int64_t u = unit0 + turn; u < unit1; u += turns) {
    const int64_t n0 = u * 32;
    if (!loaded) {
      in.load_z(p, n0, token, t);
      in.load_b(p, B, n0, 0, rank, g, t);
    }
    loaded = false;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
#pragma unroll 1
    for (int q0 = 0; q0 < groups; q0 += KG) {
      if (q0 > 0) in.load_b(p, B, n0, 16 * q0, rank, g, t);
      __syncwarp();
#pragma unroll
      for (int q = 0; q < KG; ++q) {
        if (q0 + q >= groups) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int at = (((2 * (q0 + q) + s) * mblocks + m) * 32 + lane) * 4;
          const uint4 a = *reinterpret_cast<const uint4*>(hi + at), b = *reinterpret_cast<const uint4*>(lo + at);
          const uint32_t fa[4] = {a.x, a.y, a.z, a.w}, fb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            widen<TW>(s ? in.w[q][i].y : in.w[q][i].x, b0, b1);
            mma_tf32(acc[i], fa, b0, b1);
            mma_tf32(acc[i], fb, b0, b1);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (token[h] < 0 || in.some == 0) continue;
      float v[8];
      floats8(in.z[h], p.y_type, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += acc[e >> 1][2 * h + (e & 1)];
      store8(p.y, p.y_type, token[h] * p.y_stride + in.out, in.some, p.y_vec, v);
    }
  }
  cluster_wait();
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t max_tiles(int64_t ntok, int64_t adapters) {
  return std::min(ntok, ntok / kTile + std::min(adapters, ntok) + 1);
}

bool in_pieces(const void* p, int64_t stride, int64_t bytes, int64_t piece) {
  return (uintptr_t)p % piece == 0 && stride * bytes % piece == 0;
}

template <typename TX, typename TW, int NT>
cudaError_t launch_as(const Args& a, int64_t tiles, cudaStream_t s) {
  const auto kernel = lora_kernel<TX, TW, NT>;
  const int top = (int)a.l.max_rank;
  const int smem = (kHeadInts + part_floats(top) + work_floats(top, 8 * NT)) * (int)sizeof(float);
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
cudaError_t launch_for(const Args& a, int64_t tiles, cudaStream_t s) {
  if (a.l.max_rank <= 16) return launch_as<TX, TW, 2>(a, tiles, s);
  if (a.l.max_rank <= 32) return launch_as<TX, TW, 4>(a, tiles, s);
  return launch_as<TX, TW, 8>(a, tiles, s);
}

}  // namespace

// The order of the tokens, the tiles and their number.
int64_t lora_workspace_bytes(int64_t ntok, int64_t adapters) {
  if (ntok <= kInBlock) return 0;
  return 16 + max_tiles(ntok, adapters) * 16 + ceil_div(ntok, 4) * 16;
}

cudaError_t launch_lora_add(const LoraCall& c, cudaStream_t s) {
  Args a = {};
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
  const int64_t tiles = max_tiles(c.ntok, c.lora.adapters);
  // Few tiles: several clusters share the rows of one, each with the whole of h
  // for itself, up to two thread blocks an SM, and while a block's share of B and
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
  if (c.lora.type == TQ_F16)
    return c.x_type == TQ_F32 ? launch_for<float, __half>(a, tiles, s) : launch_for<__half, __half>(a, tiles, s);
  return c.x_type == TQ_F32 ? launch_for<float, __nv_bfloat16>(a, tiles, s)
                            : launch_for<__nv_bfloat16, __nv_bfloat16>(a, tiles, s);
}

}  // namespace tq
