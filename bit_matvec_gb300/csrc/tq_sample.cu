// tq_sample.cu -- the draw of the next token: temperature, top-k, top-p, min-p
// and one given uniform number a row.
//
// A cluster of thread blocks takes a row, each a slice of it: one block where rows
// are many, sixteen where there is one. The slice stays in shared memory, or, where
// it is too large for that, in L2: logits are read from memory once, whatever the
// filters need.
//
// The kept tokens are a beginning of the order (falling logit, rising index). A
// token's place in it is an integer, its logit's bits above its complemented
// index, so each filter is a least place, the cut. A cut is found by counting
// (top-k) or weighing (top-p) the tokens in 896 ranges, first 16 to an octave
// of weight, then, where a range holds too many tokens (equal logits), equal
// parts of it, until the range around the cut holds few enough to be sorted. If
// that range and all tokens above it fit in the list, which is the rule for the
// usual settings, everything else happens on the list. Otherwise a pass over the
// slices sums the kept weights in blocks of 512 tokens, and the block that the
// draw falls into is looked through.
//
// Weights are integers (tq_weight.cuh): their sums do not depend on the order
// in which threads add. What a thread, a block of 512 tokens or the list sums up is
// in units of a weight; where such sums meet they are cut to coarse units.
//
// What bounds it: the weights' instructions, 35 a token for a row without filters. 256 rows of 262144
// take 110 us (2.4 TB/s, 2.4 instructions a cycle), 512 rows of 32768 with filters of their own 58 to 65, 64 of
// 131072 44 to 55, where top-p weighs the tokens twice and a row waits for its slowest block. Top-k alone weighs
// only the list: 200 rows of 128001 f16 58 us, in two rounds of thread blocks that each read their slice,
// wait, read it again and wait. One row of 131072 takes 15 us: five meetings of its sixteen blocks, a sort
// and the code's way into the caches.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "tq_requests.cuh"
#include "tq_weight.cuh"

namespace tq {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kIndexBits = 18;
constexpr int kList = 1024;                 // tokens that are sorted
constexpr int kBlock = 512;                 // tokens of a sum
constexpr int kMaxBlocks = kMaxVocab / kBlock + 1;
constexpr int kMaxCluster = 16;
constexpr int kSlots = 608;                 // thread blocks of a call at most: twice as many as run at once
                                            // (200 rows of 128001 f16, top-k: 46 us with 304, 58 with 608, 66
                                            // with 1216; 64 rows of 131072: 47, 55, 84. Chosen when a block's look
                                            // through its slice took longer and 200 rows took 135, 73 and 84.)
constexpr int kMaxResident = 65536;         // bytes of a slice in shared memory
static_assert(kMaxVocab == 1 << kIndexBits, "an index below a logit's bits");
static_assert(kBlock == kThreads && kList == 2 * kThreads, "one token, two entries a thread");
static_assert(kWeightBins % 128 == 0 && kWeightBins / 4 <= kThreads, "four bins a thread, in whole warps");
static_assert(kMaxBlocks <= 2 * kThreads, "two sums a thread");

using u64 = unsigned long long;
constexpr u64 kNoCut = 0;
constexpr u64 kIndexMask = (u64(1) << kIndexBits) - 1;

__device__ const ExpTable g_exp_table = make_exp_table();

struct Args {
  const void* logits;
  int64_t stride;
  int vocab, slice, cluster;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logp;
};

// Shared memory before the slice.
struct alignas(16) Shared {
  ExpTable table;
  union {
    struct {
      u64 list[kList];        // places of the tokens at a cut
      u64 weight[kList];      // (rank 0) their weights
    };
    struct {                  // while a window is narrowed: weights by bin, this block's, then (rank 0) all
      u64 mine[kWeightBins];      // coarse units, and what they lack
      uint32_t low[kWeightBins], tokens[kWeightBins];
    } by_bin;
  };
  uint32_t bins[kWeightBins]; // tokens, or leading bits of weights
  u64 sums[kMaxBlocks];       // kept weights by block, in units of a weight
  int octaves[kMaxBlocks];    // of a row without filters: what they are relative to
  u64 scan[kWarps];
  u64 give[6];                // what the other blocks of the cluster read
  u64 window[8];              // what rank 0 found
  int entry[kBlock];          // of the list, by the low bits of their indexes
  int have;                   // entries of the list
  int first;                  // lowest index of the largest logit
  u64 pick[4];
  u64 warps[3][kWeightBins / 128];
  uint32_t least_top[kWarps], tops[kThreads];   // tops: counts of threads by their largest logit
  uint32_t bound;             // a logit that so many tokens are at or above
};
static_assert(sizeof(Shared) % 16 == 0, "the slice behind it in 16-byte pieces");

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of this block's shared variable in another block of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t remote_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ u64 remote_u64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 remote_u128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void remote_put(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// The larger ones of two pairs of 16-bit values, NaN if one of the two is; a pair of minus infinities.
template <typename T> __device__ __forceinline__ uint32_t max_of_pairs(uint32_t a, uint32_t b) {
  uint32_t m;
  if (std::is_same<T, __half>::value) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
template <typename T> __device__ __forceinline__ uint32_t none_of_pairs() {
  return std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
}

// floor(a * x) of a weight sum and a float in (0, 1), exactly; `up`: the ceiling.
__device__ __noinline__ u64 fraction_of(u64 a, float x, bool up) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t mant = b >> 23 ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int shift = 150 - (int)(b >> 23 ? b >> 23 : 1);     // x = mant / 2^shift, 24 <= shift <= 149
  const u64 lo = a * mant, hi = __umul64hi(a, (u64)mant);   // below 2^88
  u64 q, left;
  if (shift < 64) {
    q = hi << (64 - shift) | lo >> shift;
    left = lo << (64 - shift);
  } else {
    const int s = shift - 64;
    q = s < 64 ? hi >> s : 0;
    left = lo | (s < 64 ? hi - (q << s) : hi);
  }
  return q + (up && left ? 1 : 0);
}

// ---------------------------------------------------------------- a thread block and its cluster
// (Functions of their own, not inlined: the kernel runs once through most of its code, and for few
// rows the time goes into fetching it.)

__device__ __forceinline__ void meet(int cluster) {
  if (cluster == 1) {
    __syncthreads();
    return;
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

struct Sum {
  u64 before, all;
};
// The sum of the threads' values before this thread, and of all.
__device__ __noinline__ Sum scan(Shared* s, u64 v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 sum = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += o;
  }
  __syncthreads();      // (the last scan's readers are done)
  if (lane == 31) s->scan[warp] = sum;
  __syncthreads();
  // every warp sums the warps' totals again
  u64 w = lane < kWarps ? s->scan[lane] : 0;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  const u64 all = __shfl_sync(0xffffffffu, w, kWarps - 1);
  const u64 before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return {(warp > 0 ? before : 0) + sum - v, all};
}
// This thread's part of its warp's sum of weights, in coarse units: the warp's sum
// is cut, not each thread's.
__device__ __forceinline__ u64 coarse(u64 units) {
  const uint32_t low = __reduce_add_sync(0xffffffffu, (uint32_t)units & ((1u << kCoarse) - 1));
  return (units >> kCoarse) + ((threadIdx.x & 31) == 0 ? low >> kCoarse : 0);
}
// The sum over the cluster of a value that all threads of a block have, by way
// of give[at], and that of the blocks before this one.
__device__ __noinline__ Sum over_cluster(Shared* s, u64 mine, int at, int cluster, int rank) {
  if (cluster == 1) {
    __syncthreads();
    return {0, mine};
  }
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s->give[at] = mine;
  meet(cluster);
  u64 v = lane < cluster ? remote_u64(remote(&s->give[at], lane)) : 0;
#pragma unroll
  for (int d = 1; d < kMaxCluster; d <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  const u64 before = __shfl_sync(0xffffffffu, v, max(rank - 1, 0));
  return {rank > 0 ? before : 0, __shfl_sync(0xffffffffu, v, kMaxCluster - 1)};
}
// Sorts the first n of kList values, falling; behind them are zeros up to the
// next power of two. A value a thread (two above 512), exchanged by shuffles
// within a warp, else through `v` and `spare` in turn, by the warps that have
// values.
__device__ __noinline__ void sort(u64* v, u64* spare, int n) {
  int size = 32;
  while (size < n) size *= 2;
  const int threads = min(size, kThreads), i = threadIdx.x;
  const bool two = size > kThreads;
  if (i < threads) {
    u64 x = v[i], y = two ? v[i + kThreads] : 0;
    u64* from = spare;
    u64* next = v;
#pragma unroll 1
    for (int k = 2; k <= size; k *= 2)
#pragma unroll 1
      for (int j = k / 2; j > 0; j /= 2) {
        if (j == kThreads) {               // the whole, falling: a thread's two
          const u64 a = max(x, y);
          y = min(x, y);
          x = a;
          continue;
        }
        u64 p, q = 0;
        if (j < 32) {
          p = __shfl_xor_sync(0xffffffffu, x, j);
          if (two) q = __shfl_xor_sync(0xffffffffu, y, j);
        } else {
          from[i] = x;
          if (two) from[i + kThreads] = y;
          named_barrier_sync(1, threads);
          p = from[i ^ j];
          if (two) q = from[(i ^ j) + kThreads];
          u64* const t = from;
          from = next;
          next = t;
        }
        const bool low = (i & j) == 0;
        x = low == ((i & k) == 0) ? max(x, p) : min(x, p);
        if (two) y = low == (((i + kThreads) & k) == 0) ? max(y, q) : min(y, q);
      }
    named_barrier_sync(1, threads);        // (the last exchange through memory is read)
    v[i] = x;
    if (two) v[i + kThreads] = y;
  }
  __syncthreads();
}

struct Window {
  u64 lo, hi;       // places
  u64 above;        // tokens above it (a narrowed one by weight: what they weigh, in coarse units)
  u64 inside;       // tokens in it, at most
  u64 upto;         // tokens in it or above, at most
};

// By one warp: the first of kWeightBins values v for which above + the sum up to
// it reaches `target` (kWeightBins if none does), and what is before it.
struct Found {
  int bin;
  u64 before;
};
__device__ __noinline__ Found first_reaching(const u64* v, u64 target, u64 above) {
  constexpr int kEach = kWeightBins / 32;
  static_assert(kEach <= 32, "a bin of a lane's share a lane");
  const int lane = threadIdx.x & 31;
  u64 sum = 0;
#pragma unroll 8
  for (int e = 0; e < kEach; ++e) sum += v[lane * kEach + (e + lane) % kEach];   // (no two lanes in one bank)
  u64 upto = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  const unsigned m = __ballot_sync(0xffffffffu, above + upto >= target);
  if (m == 0) return {kWeightBins, above + __shfl_sync(0xffffffffu, upto, 31)};
  const int share = __ffs(m) - 1;
  const u64 base = above + __shfl_sync(0xffffffffu, upto - sum, share);
  const u64 x = lane < kEach ? v[share * kEach + lane] : 0;
  upto = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  const int at = __ffs(__ballot_sync(0xffffffffu, base + upto >= target)) - 1;
  return {share * kEach + at, base + __shfl_sync(0xffffffffu, upto - x, at)};
}
template <typename T> struct Row {
  Shared* s;
  const T* xs;                // this block's slice: values pad .. end - 1 from here
  int cluster, rank;
  int start;                  // the token of xs[0]
  int pad, end, blocks;       // blocks of 512 values that hold some
  bool infinite;              // a plus infinity: every other logit is minus infinity beside it
  Weigher weigh;

  __device__ __forceinline__ u64 place(float l, int i) const {   // i: in xs
    return ((u64)order_key(l) << kIndexBits) | (unsigned)(kMaxVocab - 1 - (start + i));
  }
  __device__ __forceinline__ float beside_infinity(float l) const { return l == INFINITY ? 0.0f : -INFINITY; }
  // One logit, NaN outside the slice.
  __device__ __forceinline__ float value(int i) const {
    if (i < pad || i >= end) return NAN;
    const float l = Elem<T>::up(xs[i]);
    return infinite ? beside_infinity(l) : l;
  }
  // Calls f(four logits, the index of the first in xs) for every token (NaN for
  // what is none); a warp's turn is a block of 512, after which done(block).
  template <typename F, typename D> __device__ __forceinline__ void each(F f, D done) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int b = warp; b < blocks; b += kWarps) {
      const int i0 = b * kBlock + lane * 4;
      Vec<T, 4> v[4];
      const bool whole = b * kBlock >= pad && (b + 1) * kBlock <= end;
      if (whole) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const Vec<T, 4>*>(xs + i0 + j * 128);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int i = i0 + (e >> 2) * 128 + (e & 3);
          v[e >> 2].v[e & 3] = i >= pad && i < end ? xs[i] : Elem<T>::down(NAN);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) l[e] = Elem<T>::up(v[j].v[e]);
        if (infinite) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (l[e] == l[e]) l[e] = beside_infinity(l[e]);
        }
        f(l, i0 + j * 128);
      }
      done(b);
    }
  }
  template <typename F> __device__ __forceinline__ void each(F f) const {
    each(f, [](int) {});
  }
  // The sum of the weights of four tokens that fulfil `counts`.
  template <typename C> __device__ __forceinline__ u64 weigh_if(const float (&l)[4], C counts) const {
    bool in[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) in[e] = counts(e);
    if (!__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) return 0;
    uint64_t w[4];
    int bits[4];
    weigh(l, w, bits);
    u64 sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += in[e] ? w[e] : 0;
    return sum;
  }

  // ---- finding a cut

  // By one warp: the least place of a weight's bin of at most b.
  __device__ __forceinline__ u64 bin_end(int b, uint32_t top_key) const {
    const uint32_t lane = threadIdx.x & 31;
    // Where the exponent passes the bin's end, to a few steps of a float: half a
    // step of 2^-11 below the multiple that begins it.
    const float edge = __int_as_float(((Weigher::kMagic >> Weigher::kBinShift) - b) << Weigher::kBinShift);
    const float guess = __fdiv_rn((edge - 0x1p-12f) - weigh.k, weigh.c_hi) + weigh.shift;
    if (weigh.bin(key_value(top_key)) > b) return (u64)(top_key + 1) << kIndexBits;   // above all tokens
    uint32_t lo = 0, hi = top_key;         // (whose bin is at most b)
    const uint32_t near = order_key(guess);
    if (top_key > 31) {
      const uint32_t base = min(near - min(near, 16u), top_key - 31);
      const unsigned m = __ballot_sync(0xffffffffu, weigh.bin(key_value(base + lane)) <= b);
      if (m != 0 && !(m & 1u)) lo = hi = base + (__ffs(m) - 1);
    }
    // otherwise the least key whose bin is at most b, 32 candidates a step
    while (lo < hi) {
      const uint32_t step = (hi - lo) / 32 + 1, at = lo + lane * step;
      const bool in = at < hi && weigh.bin(key_value(at)) <= b;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (m) {
        const uint32_t l = __ffs(m) - 1;
        hi = lo + l * step;
        lo = l > 0 ? lo + (l - 1) * step + 1 : hi;
      } else {
        lo += min(31u, (hi - 1 - lo) / step) * step + 1;    // behind the last candidate below hi
      }
    }
    return (u64)lo << kIndexBits;
  }

  // A word of what rank 0 found, for all blocks: by one warp.
  __device__ __forceinline__ void publish(int word, u64 v) const {
    const int lane = threadIdx.x & 31;
    if (lane < cluster) remote_put(remote(&s->window[word], lane), v);
  }
  __device__ __forceinline__ Window published(u64& target) const {
    meet(cluster);
    target = s->window[5];
    return {s->window[0], s->window[1], s->window[2], s->window[3], s->window[4]};
  }

  // The range around the cut, of tokens from `from` on: by count, the least
  // place such that `target` tokens are at it or above, none of which is below
  // `least_top`; by weight, such that they weigh the share `share` of all at
  // least (`target` becomes that, in coarse units). The bins are zeros.
  __device__ __forceinline__ Window search(bool by_weight, u64& target, u64 from, uint32_t top_key, float share,
                                           float least_top) const {
    const int tid = threadIdx.x;
    // (tokens that weigh nothing do not help to reach a weight)
    Window w = {max(from, (u64)order_key(by_weight ? weigh.least : least_top) << kIndexBits),
                ((u64)top_key << kIndexBits) | kIndexMask, 0, 0, 0};
    if (by_weight) {
      u64 mine = 0;
      const float lo = fmaxf(weigh.least, key_value(max((uint32_t)(from >> kIndexBits), order_key(-INFINITY))));
      each([&](const float (&l)[4], int i) {
        bool in[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) in[e] = l[e] >= lo && (l[e] > lo || place(l[e], i + e) >= from);
        if (!__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) return;
        uint64_t wt[4];
        int bits[4];
        uint32_t lead[4];
        weigh(l, wt, bits, lead);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (in[e]) {
            mine += wt[e];
            atomicAdd(&s->bins[Weigher::bin_of(bits[e])], lead[e]);
          }
      });
      const u64 sum = scan(s, coarse(mine)).all;
      if (tid == 0) s->give[0] = sum;
    } else {
      each([&](const float (&l)[4], int) {
        if (fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= least_top) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (l[e] >= least_top) atomicAdd(&s->bins[weigh.bin(l[e])], 1u);
        }
      });
    }
    meet(cluster);
    if (rank == 0) {
      const int lane = tid & 31, warp = tid >> 5;
      if (by_weight) {
        u64 all = lane < cluster ? remote_u64(remote(&s->give[0], lane)) : 0;
#pragma unroll
        for (int d = kMaxCluster / 2; d > 0; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
        all = __shfl_sync(0xffffffffu, all, 0);
        target = share > 0.0f ? max(u64(1), fraction_of(all, share, true)) : 1;
      }
      // This thread's four bins, of all blocks: tokens (at most), and what
      // counts, at least and at most; and the sums before them.
      u64 n[4] = {0, 0, 0, 0}, lo[4], hi[4], at_lo = 0, at_hi = 0, at_n = 0;
      if (tid < kWeightBins / 4) {
        for (int r0 = 0; r0 < cluster; r0 += 8) {
          uint4 v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            v[r] = r0 + r < cluster ? remote_u128(remote(&s->bins[4 * tid], r0 + r)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            n[0] += v[r].x;
            n[1] += v[r].y;
            n[2] += v[r].z;
            n[3] += v[r].w;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = hi[e] = n[e];
          if (by_weight) {
            // Sums of weights' first 13 bits, 2^12 - 1 at least (just below a
            // power of two the table's entry is that power's): a token for each of
            // these in the sum, at most, each cut by less than one, and to a unit.
            const int shift = 34 - Weigher::octave_of(4 * tid + e);
            auto shifted = [&](u64 v) { return shift >= 0 ? v << shift : v >> -shift; };
            const u64 most = (n[e] + (n[e] >> 11)) >> 12, v = shifted(n[e]);
            lo[e] = v - min(v, most);
            hi[e] = most ? shifted(n[e] + most) + most + 1 : 0;
            n[e] = most;
          }
        }
        const u64 sum_lo = lo[0] + lo[1] + lo[2] + lo[3], sum_hi = hi[0] + hi[1] + hi[2] + hi[3];
        const u64 sum_n = n[0] + n[1] + n[2] + n[3];
        at_lo = sum_lo;
        at_hi = sum_hi;
        at_n = sum_n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const u64 x = __shfl_up_sync(0xffffffffu, at_lo, d);
          if (lane >= d) at_lo += x;
          if (by_weight) {
            const u64 y = __shfl_up_sync(0xffffffffu, at_hi, d), z = __shfl_up_sync(0xffffffffu, at_n, d);
            if (lane >= d) {
              at_hi += y;
              at_n += z;
            }
          }
        }
        if (!by_weight) at_hi = at_n = at_lo;
        if (lane == 31) {
          s->warps[0][warp] = at_lo;
          s->warps[1][warp] = at_hi;
          s->warps[2][warp] = at_n;
        }
        at_lo -= sum_lo;
        at_hi -= sum_hi;
        at_n -= sum_n;
      }
      if (tid == kThreads - 1) {
        s->pick[0] = 0;
        s->pick[1] = kWeightBins;
        s->pick[2] = 0;
      }
      __syncthreads();
      u64 tokens = 0;
      if (tid < kWeightBins / 4) {
        for (int w = 0; w < kWeightBins / 128; ++w) {
          tokens += s->warps[2][w];
          if (w >= warp) continue;
          at_lo += s->warps[0][w];
          at_hi += s->warps[1][w];
          at_n += s->warps[2][w];
        }
        if (tid == 0) s->pick[3] = tokens;
      }
      __syncthreads();
      if (tid < kWeightBins / 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (at_hi < target && at_hi + hi[e] >= target) {      // the first that may reach the target
            s->pick[0] = 4 * tid + e;
            s->pick[2] = at_n;
          }
          if (at_lo < target && at_lo + lo[e] >= target) {      // the first that surely does
            s->pick[1] = 4 * tid + e;
            s->pick[3] = at_n + n[e];
          }
          at_lo += lo[e];
          at_hi += hi[e];
          at_n += n[e];
        }
      }
      __syncthreads();
      if (warp == 0) {
        const int last = (int)s->pick[1];
        publish(0, max(w.lo, last < kWeightBins ? bin_end(last, top_key) : 0));
        publish(2, s->pick[2]);
        publish(3, s->pick[3] - s->pick[2]);
      } else if (warp == 1) {
        const int first = (int)s->pick[0];
        publish(1, first > 0 ? min(w.hi, bin_end(first - 1, top_key) - 1) : w.hi);
        publish(4, s->pick[3]);
        publish(5, target);
      }
    }
    return published(target);
  }

  // Narrows a window until at most kList tokens are inside: equal parts of it,
  // with exact sums. (Not inlined, and given a copy of the row: it is for many
  // equal logits, and for many tokens that weigh next to nothing.)
  static __device__ __noinline__ Window narrow(Row row, Window w, bool by_weight, u64 target) {
    Shared* const s = row.s;
    const int tid = threadIdx.x;
    u64* const sums = s->by_bin.mine;
    uint32_t* const low = s->by_bin.low;
    uint32_t* const tokens = s->by_bin.tokens;
    while (w.inside > kList) {
      int shift = 0;
      while (((w.hi - w.lo) >> shift) >= kWeightBins) ++shift;
      meet(row.cluster);
      for (int j = tid; j < kWeightBins; j += kThreads) {
        s->bins[j] = 0;
        sums[j] = 0;
        low[j] = 0;
      }
      __syncthreads();
      u64 above = 0;
      row.each([&](const float (&l)[4], int i) {
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          const float x = e == 0 ? l[0] : e == 1 ? l[1] : e == 2 ? l[2] : l[3];
          if (!(x == x)) continue;
          const u64 q = row.place(x, i + e);
          const bool weighs = by_weight && x >= row.weigh.least;
          if (q > w.hi) {
            above += by_weight ? (weighs ? row.weigh.one(x) : 0) : 1;
          } else if (q >= w.lo) {
            const int j = (int)((w.hi - q) >> shift);
            atomicAdd(&s->bins[j], 1u);
            if (weighs) {
              const u64 units = row.weigh.one(x);
              atomicAdd(&sums[j], units >> kCoarse);
              atomicAdd(&low[j], (uint32_t)units & ((1u << kCoarse) - 1));
            }
          }
        }
      });
      __syncwarp();
      above = over_cluster(s, scan(s, by_weight ? coarse(above) : above).all, 1, row.cluster, row.rank).all;
      if (row.rank == 0) {
        for (int j = tid; j < kWeightBins; j += kThreads) {
          uint32_t n = 0, lack = 0;
          u64 v = 0;
          for (int r = 0; r < row.cluster; ++r) {
            n += remote_u32(remote(&s->bins[j], r));
            if (by_weight) {
              v += remote_u64(remote(&sums[j], r));
              lack += remote_u32(remote(&low[j], r));
            }
          }
          tokens[j] = n;
          sums[j] = by_weight ? v + (lack >> kCoarse) : n;
        }
        __syncthreads();
        if (tid < 32) {
          const Found at = first_reaching(sums, target, above);
          const int bin = min(at.bin, kWeightBins - 1);
          const u64 top = w.hi;
          w.hi = top - ((u64)bin << shift);
          w.lo = max(w.lo, top - min(top, ((u64)(bin + 1) << shift) - 1));
          w.above = at.before;
          w.inside = tokens[bin];
          row.publish(0, w.lo);
          row.publish(1, w.hi);
          row.publish(2, w.above);
          row.publish(3, w.inside);
        }
      }
      w = row.published(target);
    }
    return w;
  }

  // The tokens of the window in this block's list. `weights`: the sum of the
  // weights of those above it is returned, in coarse units, and by block in s->sums.
  __device__ __forceinline__ u64 gather(const Window& w, bool weights) const {
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) s->have = 0;
    __syncthreads();
    const float lo = key_value(max((uint32_t)(w.lo >> kIndexBits), order_key(-INFINITY)));
    const float hi = key_value((uint32_t)(w.hi >> kIndexBits));
    auto collect = [&](float l, int i) {
      const u64 q = place(l, i);
      if (q < w.lo || q > w.hi) return;
      const int at = atomicAdd(&s->have, 1);
      if (at < kList) s->list[at] = q;
    };
    if (!weights) {
      each([&](const float (&l)[4], int i) {
        if (fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= lo) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (l[e] >= lo) collect(l[e], i + e);
        }
      });
      __syncthreads();
      return 0;
    }
    u64 mine = 0, all = 0;
    each([&](const float (&l)[4], int i) {
      bool at_window = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) at_window |= l[e] >= lo && l[e] <= hi;
      if (at_window) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (l[e] >= lo && l[e] <= hi) collect(l[e], i + e);
      }
      __syncwarp();
      mine += weigh_if(l, [&](int e) { return l[e] >= hi && (l[e] > hi || place(l[e], i + e) > w.hi); });
    }, [&](int b) {
      all += mine;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
      if (lane == 0) s->sums[b] = mine;
      mine = 0;
    });
    return scan(s, coarse(all)).all;
  }

  // The tokens at `lo` or above in this block's list: each warp's in a part of
  // s->weight first. s->have is more than kList if they do not fit there.
  __device__ __forceinline__ void gather_from(float lo) const {
    constexpr int kEach = kList / kWarps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = 0;
    each([&](const float (&l)[4], int i) {
      if (!__any_sync(0xffffffffu, fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= lo)) return;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned m = __ballot_sync(0xffffffffu, l[e] >= lo);
        const int at = n + __popc(m & ((1u << lane) - 1));
        if (l[e] >= lo && at < kEach) s->weight[warp * kEach + at] = place(l[e], i + e);
        n += __popc(m);
      }
    });
    if (lane == 0) s->least_top[warp] = (uint32_t)n;
    __syncthreads();
    const uint32_t of = lane < kWarps ? s->least_top[lane] : 0;
    const bool fits = __all_sync(0xffffffffu, of <= kEach);
    const int all = (int)__reduce_add_sync(0xffffffffu, of);
    const int before = (int)__reduce_add_sync(0xffffffffu, lane < warp ? of : 0);
    if (fits)
      for (int i = lane; i < n; i += 32) s->list[before + i] = s->weight[warp * kEach + i];
    if (threadIdx.x == 0) s->have = fits ? all : kList + 1;
  }
  // Entries of all blocks' lists (after the cluster has met).
  __device__ __forceinline__ int listed() const {
    const int lane = threadIdx.x & 31;
    return (int)__reduce_add_sync(0xffffffffu, lane < cluster ? remote_u32(remote(&s->have, lane)) : 0);
  }

  // (rank 0) All blocks' lists in this one's, sorted, the highest first; returns
  // their number. The weights are in s->weight.
  __device__ __forceinline__ int join() const {
    const int tid = threadIdx.x, lane = tid & 31;
    __syncthreads();
    int have = lane < cluster ? (int)remote_u32(remote(&s->have, lane)) : 0;
    const int mine = __shfl_sync(0xffffffffu, have, 0);
    int upto = have;      // entries of the blocks up to the lane's
#pragma unroll
    for (int d = 1; d < kMaxCluster; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const int n = min(__shfl_sync(0xffffffffu, upto, kMaxCluster - 1), kList);
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) {
      const int at = mine + j * kThreads + tid;
      // the block that has entry `at`: the first whose entries reach beyond it
      int r = 0, base = 0;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        const int e = __shfl_sync(0xffffffffu, upto, c);
        if (e <= at) {
          r = c + 1;
          base = e;
        }
      }
      if (at < kList) s->list[at] = at < n ? remote_u64(remote(&s->list[at - base], r)) : 0;
    }
    __syncthreads();
    sort(s->list, s->weight, n);
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) {
      const int i = tid + j * kThreads;
      const float l = key_value((uint32_t)(s->list[i] >> kIndexBits));
      s->weight[i] = i < n && l >= weigh.least ? weigh.one(l) : 0;
    }
    __syncthreads();
    return n;
  }
  // (rank 0) The sums of the sorted weights up to each entry, in `sums`.
  __device__ __forceinline__ void sum_up(u64* sums) const {
    const int i = 2 * threadIdx.x;
    const u64 x = s->weight[i], y = s->weight[i + 1], at = scan(s, x + y).before;
    sums[i] = at + x;
    sums[i + 1] = at + x + y;
    __syncthreads();
  }
};

// (rank 0) The number of entries for which `counts` holds.
template <typename C> __device__ __forceinline__ int count_of(C counts) {
  const int i = threadIdx.x;
  return __syncthreads_count(counts(i)) + __syncthreads_count(counts(i + kThreads));
}

// The place of the draw among weights that sum to `total`.
__device__ __forceinline__ u64 goal_of(u64 total, float u) {
  return u > 0.0f ? (u < 1.0f ? min(fraction_of(total, u, false), total - 1) : total - 1) : 0;
}

__device__ __noinline__ void answer(const Args& a, Weigher weigh, int64_t row, int token, float l, u64 total,
                                    bool alone) {
  a.tokens[row] = token;
  if (a.logp) a.logp[row] = alone ? 0.0f : weigh.log_share(l, total);
}

// (rank 0) The draw from a sorted list whose first `kept` entries are the kept
// tokens: the sums of their weights by the upper half of their indexes, then, for
// the part that the draw falls into, by index. bins: room for 512 values.
__device__ __noinline__ void draw_from_list(Shared* s, u64* bins, const Args& a, Weigher weigh, int64_t row, int kept,
                                            u64 total, float u) {
  const int tid = threadIdx.x;
  static_assert(kIndexBits == 18 && kThreads == 512 && kBlock == 512, "two halves of 9 bits");
  u64 goal = goal_of(total, u);
  int part = 0;
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    bins[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) {
      const int i = tid + j * kThreads;
      if (i >= kept) continue;
      const int index = kMaxVocab - 1 - (int)(s->list[i] & kIndexMask);
      if (half == 0) {
        atomicAdd(&bins[index >> 9], s->weight[i]);
      } else if (index >> 9 == part) {
        bins[index & 511] = s->weight[i];
        s->entry[index & 511] = i;
      }
    }
    __syncthreads();
    const u64 mine = bins[tid], at = scan(s, mine).before;
    if (at <= goal && goal < at + mine) {
      if (half == 0) {
        s->pick[0] = tid;
        s->pick[1] = at;
      } else {
        const u64 e = s->list[s->entry[tid]];
        answer(a, weigh, row, part << 9 | tid, key_value((uint32_t)(e >> kIndexBits)), total >> kCoarse, mine == total);
      }
    }
    __syncthreads();
    part = (int)s->pick[0];
    goal -= s->pick[1];
  }
}

// A row without filters, in one pass over its logits as they come from memory:
// the weights of a block of 512 tokens are relative to its own largest logit, in
// whole octaves, so that sums join by shifts. False if the row needs the other
// way: an infinite logit, or a temperature so low that exponents pass 2000.
template <typename T>
__device__ __noinline__ bool draw_unfiltered(Shared* s, const Args& a, const T* from16, Row<T> r, int64_t row, float t,
                                             float u) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kNone = -(1 << 20);         // octave of a block without a logit above minus infinity
  enum { kNan = 1, kOther = 2 };
  r.weigh.set_temperature(t);
  r.weigh.set_octave(0.0f, &s->table);      // (a warp may have no block of its own)
  int flags = 0;
#pragma unroll 1
  for (int b = warp; b < r.blocks; b += kWarps) {
    float l[16];
    const int i0 = b * kBlock + lane * 4;
    if (b * kBlock >= r.pad && (b + 1) * kBlock <= r.end) {
      Vec<T, 4> v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const Vec<T, 4>*>(from16 + i0 + j * 128);
#pragma unroll
      for (int e = 0; e < 16; ++e) l[e] = Elem<T>::up(v[e >> 2].v[e & 3]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int i = i0 + (e >> 2) * 128 + (e & 3);
        l[e] = i >= r.pad && i < r.end ? Elem<T>::up(from16[i]) : -INFINITY;
      }
    }
    float top = l[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) top = max_or_nan(top, l[e]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    u64 sum = 0;
    int octave = kNone;
    if (top != top) {
      flags |= kNan;
    } else if (top != -INFINITY) {
      if (top == INFINITY || !(fabsf(top * r.weigh.c_hi) < 1900.0f)) {
        flags |= kOther;
      } else {
        octave = r.weigh.set_octave(top, &s->table);
        const float least = (float)(octave - kOctaves) / r.weigh.c_hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x[4] = {l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]};
          uint64_t w[4];
          int bits[4];
          r.weigh(x, w, bits);
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += x[e] >= least ? w[e] : 0;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      }
    }
    if (lane == 0) {
      s->sums[b] = sum;
      s->octaves[b] = octave;
    }
  }
  // ---- this block's sum, and the cluster's
  if (tid == 0) s->have = 0;
  __syncthreads();
  if (flags && lane == 0) atomicOr(&s->have, flags);
  const int b0 = 2 * tid, b1 = b0 + 1;
  int top = max(b0 < r.blocks ? s->octaves[b0] : kNone, b1 < r.blocks ? s->octaves[b1] : kNone);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s->least_top[warp] = (uint32_t)top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, (int)s->least_top[lane & (kWarps - 1)]);
  auto shifted = [](u64 v, int by) { return by < 64 ? v >> by : 0; };
  const u64 block0 = b0 < r.blocks ? shifted(s->sums[b0], top - s->octaves[b0] + kCoarse) : 0;
  const u64 block1 = b1 < r.blocks ? shifted(s->sums[b1], top - s->octaves[b1] + kCoarse) : 0;
  const Sum blocks = scan(s, block0 + block1);
  if (tid == 0) {
    s->give[4] = blocks.all;
    s->give[5] = (u64)(uint32_t)top << 32 | (uint32_t)s->have;
  }
  meet(r.cluster);
  u64 v = 0, what = (u64)(uint32_t)kNone << 32;
  if (lane < r.cluster) {
    v = remote_u64(remote(&s->give[4], lane));
    what = remote_u64(remote(&s->give[5], lane));
  }
  const int octave = (int)(what >> 32);
  const int highest = __reduce_max_sync(0xffffffffu, octave);
  flags = (int)__reduce_or_sync(0xffffffffu, (uint32_t)what);
  if (flags & kNan) flags = kNan;
  if (flags == kOther) return false;
  if (flags == kNan || highest == kNone) {
    if (r.rank == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.logp) a.logp[row] = NAN;
    }
    return true;
  }
  v = shifted(v, highest - octave);
  u64 upto = v;
#pragma unroll
  for (int d = 1; d < kMaxCluster; d <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  const u64 total = __shfl_sync(0xffffffffu, upto, kMaxCluster - 1);
  const u64 before = __shfl_sync(0xffffffffu, upto - v, r.rank), mine = __shfl_sync(0xffffffffu, v, r.rank);
  const u64 goal = goal_of(total, u);
  if (!(before <= goal && goal < before + mine)) return true;       // (the same for all threads of a block)
  // ---- the goal in this block's units, then in those of the 512 tokens it falls into
  const u64 here = min((goal - before) << (highest - top), blocks.all - 1);
  if (blocks.before <= here && here < blocks.before + block0 + block1) {
    const bool second = here >= blocks.before + block0;
    const int b = second ? b1 : b0;
    s->pick[0] = b;
    s->pick[1] = min((here - blocks.before - (second ? block0 : 0)) << (top - s->octaves[b] + kCoarse), s->sums[b] - 1);
  }
  __syncthreads();
  const int b = (int)s->pick[0], i = b * kBlock + tid;
  r.weigh.k = 6144.0f - (float)s->octaves[b];
  const float l = i >= r.pad && i < r.end ? Elem<T>::up(from16[i]) : -INFINITY;
  const u64 w = l >= (float)(s->octaves[b] - kOctaves) / r.weigh.c_hi ? r.weigh.one(l) : 0;
  const u64 at = scan(s, w).before;
  if (at <= s->pick[1] && s->pick[1] < at + w) {
    r.weigh.k = 6144.0f - (float)highest;      // what the total is relative to
    answer(a, r.weigh, row, r.start + i, l, total, shifted(w, highest - s->octaves[b] + kCoarse) == total);
  }
  return true;
}

template <typename T, bool kResident>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared* const s = reinterpret_cast<Shared*>(raw);
  unsigned char* const room = raw + sizeof(Shared);     // the slice, or 16 KB
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  const int64_t row = blockIdx.x / a.cluster;
  for (int j = tid; j < (int)(sizeof(ExpTable) / 16); j += kThreads)
    reinterpret_cast<uint4*>(&s->table)[j] = reinterpret_cast<const uint4*>(&g_exp_table)[j];
  for (int j = tid; j < kWeightBins; j += kThreads) s->bins[j] = 0;
  s->tops[tid] = 0;
  if (tid == 0) {
    s->first = 0x7fffffff;
    s->bound = 0xffffffffu;
  }
  pdl_wait_primary();
  pdl_launch_dependents();

  const float temp = a.temperature ? a.temperature[row] : 1.0f;
  const float p = a.top_p ? a.top_p[row] : 1.0f, mp = a.min_p ? a.min_p[row] : 0.0f, u = a.u[row];
  const int k = mp > 1.0f ? 1 : a.top_k ? a.top_k[row] : 0;     // (no weight is above 1: one token, the first)
  const float t = fminf(temp, 0x1p100f);
  const bool by_count = k > 0 && k < a.vocab, by_weight = p < 1.0f;
  const int from = rank * a.slice, count = max(0, min(a.slice, a.vocab - from));
  const T* const x = static_cast<const T*>(a.logits) + row * a.stride + from;
  // in shared memory as it lies in memory within 16 bytes, so that whole pieces are copied
  constexpr int kPiece = 16 / (int)sizeof(T);
  const int pad = (int)((uintptr_t)x % 16 / sizeof(T)), end = pad + count;
  Row<T> r = {s, kResident ? reinterpret_cast<const T*>(room) : x - pad, a.cluster, rank, from - pad, pad, end,
              count > 0 ? (end + kBlock - 1) / kBlock : 0, false, {}};
  if (temp >= 0x1p-100f && temp < INFINITY && !by_count && !by_weight && !(mp > 0.0f)) {
    __syncthreads();
    const bool done = draw_unfiltered<T>(s, a, x - pad, r, row, t, u);
    meet(a.cluster);          // what the other blocks read is read
    if (done) return;
  }

  // ---- the slice, its largest logit, and whether there is a NaN
  float top = -INFINITY;
  {
    const uint4* const from16 = reinterpret_cast<const uint4*>(x - pad);
    const int first = pad ? 1 : 0, last = end / kPiece;        // whole pieces
    uint32_t pairs = none_of_pairs<T>();                       // 16-bit types: two maxima in one operation
#pragma unroll 4
    for (int i = first + tid; i < last; i += kThreads) {
      const uint4 q = ldg_stream_v4(from16 + i);
      if (kResident) reinterpret_cast<uint4*>(room)[i] = q;
      if constexpr (sizeof(T) == 2) {
        pairs = max_of_pairs<T>(pairs, max_of_pairs<T>(max_of_pairs<T>(q.x, q.y), max_of_pairs<T>(q.z, q.w)));
      } else {
        top = max_or_nan(max_or_nan(top, max_or_nan(__uint_as_float(q.x), __uint_as_float(q.y))),
                         max_or_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
      }
    }
    if constexpr (sizeof(T) == 2) {
      const Vec<T, 2> v = *reinterpret_cast<const Vec<T, 2>*>(&pairs);
      top = max_or_nan(Elem<T>::up(v.v[0]), Elem<T>::up(v.v[1]));
    }
    // the ends: before the first whole piece, behind the last one
    const int head = min(end, first * kPiece), tail = max(head, last * kPiece);
    const int i = tid < kPiece ? pad + tid : tail + tid - kPiece;
    if (tid < 2 * kPiece && (tid < kPiece ? i < head : i < end)) {
      const T v = x[i - pad];
      if (kResident) reinterpret_cast<T*>(room)[i] = v;
      top = max_or_nan(top, Elem<T>::up(v));
    }
  }
  // `top` is each thread's largest logit now. As many threads as have theirs at
  // or above some value, so many tokens are there; the `share`-th largest of them
  // bounds a cut by count from below (and few tokens are above it that do not
  // belong). It is found among 512 equal parts of their range.
  uint32_t bound = 0;
  const int share = (k + a.cluster - 1) / a.cluster;
  const bool bounded = by_count && share <= kThreads;
  {
    const float own = top;
    uint32_t least = __reduce_min_sync(0xffffffffu, order_key(top));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    float* const tops = reinterpret_cast<float*>(s->scan);
    if (lane == 0) {
      tops[warp] = top;
      s->least_top[warp] = least;
    }
    __syncthreads();
    top = tops[lane & (kWarps - 1)];
    least = __reduce_min_sync(0xffffffffu, s->least_top[lane & (kWarps - 1)]);
#pragma unroll
    for (int d = kWarps / 2; d > 0; d >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (bounded) {
      const float low = key_value(least);
      const float steps = (float)(kThreads - 1) / (top - low);      // (no number where the range is infinite or nothing)
      const int part = min(kThreads - 1, max(0, (int)((own - low) * steps)));
      atomicAdd(&s->tops[part], 1u);
      __syncthreads();
      // every warp: 16 parts a lane, the highest first
      uint32_t n = 0;
      constexpr int kEach = kThreads / 32;
#pragma unroll
      for (int e = 0; e < kEach; ++e) n += s->tops[kThreads - 1 - (lane * kEach + e)];
      uint32_t upto = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      const int lane_of = __ffs(__ballot_sync(0xffffffffu, upto >= (uint32_t)share)) - 1;
      uint32_t before = __shfl_sync(0xffffffffu, upto - n, lane_of);
      int at = kThreads - 1 - lane_of * kEach;
      for (; (before += s->tops[at]) < (uint32_t)share; --at) {
      }
      // the least of the threads' values in that part or above
      const uint32_t mine = __reduce_min_sync(0xffffffffu, part >= at ? order_key(own) : 0xffffffffu);
      if (lane == 0) atomicMin(&s->bound, mine);
      __syncthreads();
      bound = s->bound;
    }
    if (a.cluster > 1) {
      if (tid == 0) s->give[3] = (u64)bound << 32 | __float_as_uint(top);
      meet(a.cluster);
      const u64 v = remote_u64(remote(&s->give[3], min(lane, a.cluster - 1)));
      top = __uint_as_float((uint32_t)v);
      bound = __reduce_min_sync(0xffffffffu, (uint32_t)(v >> 32));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
  }
  if (top != top || top == -INFINITY || !(temp >= 0.0f) || temp == INFINITY) {
    if (rank == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.logp) a.logp[row] = NAN;
    }
  } else if (temp < 0x1p-100f) {
    int first = 0x7fffffff;
    r.each([&](const float (&l)[4], int i) {
#pragma unroll
      for (int e = 3; e >= 0; --e)
        if (l[e] == top) first = min(first, r.start + i + e);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) atomicMin(&s->first, first);
    meet(a.cluster);
    if (rank == 0 && warp == 0) {
      first = lane < a.cluster ? (int)remote_u32(remote(&s->first, lane)) : 0x7fffffff;
      first = __reduce_min_sync(0xffffffffu, first);
      if (lane == 0) {
        a.tokens[row] = first;
        if (a.logp) a.logp[row] = 0.0f;
      }
    }
  } else {
    r.infinite = top == INFINITY;
    if (r.infinite) top = 0.0f;
    r.weigh.set_temperature(t);
    r.weigh.set_top(top, t, &s->table);
    const uint32_t top_key = order_key(top);
    u64 floor = kNoCut;       // of min-p
    if (mp > 0.0f) {
      // the least float that is top + T ln(min-p) or above: the sum, and one up if it was rounded down
      float hi, lo;
      scaled_log(mp, t, s->table, hi, lo);
      const float sum = __fadd_rn(top, hi), b = __fsub_rn(sum, top);
      const float off = __fadd_rn(__fadd_rn(__fsub_rn(top, __fsub_rn(sum, b)), __fsub_rn(hi, b)), lo);
      const uint32_t key = hi < 0.0f ? order_key(sum) + (off > 0.0f ? 1u : 0u) : top_key;
      floor = (u64)min(key, top_key) << kIndexBits;
    }
    bool drawn = false;       // by rank 0, from the list
    bool summed = false;      // s->sums holds the kept weights
    u64 cut = kNoCut;
#pragma unroll 1
    for (int which = by_count ? 0 : 1; which < (by_weight ? 2 : 1) && !drawn; ++which) {
      const bool weights = which == 1;
      if (weights && by_count) {      // the bins are in use no more, and zeros again
        meet(a.cluster);
        for (int j = tid; j < kWeightBins; j += kThreads) s->bins[j] = 0;
        __syncthreads();
      }
      u64 target = (u64)k, above = 0;
      Window w = {0, ((u64)top_key << kIndexBits) | kIndexMask, 0, 0, 0};
      bool whole = false;       // all tokens that may be kept are in the list
      const bool usable = bounded && !r.infinite && bound > order_key(-INFINITY);
      if (!weights && usable) {
        r.gather_from(key_value(bound));
        meet(a.cluster);
        whole = r.listed() <= kList;
        if (!whole) meet(a.cluster);       // the last reading of the counts is over
      }
      if (!whole) {
        w = r.search(weights, target, cut, top_key, p, usable ? key_value(bound) : -INFINITY);
        whole = w.upto <= kList;
        if (whole) w.hi = ((u64)top_key << kIndexBits) | kIndexMask;
        else if (w.inside > kList) w = Row<T>::narrow(r, w, weights, target);
        const u64 mine = r.gather(w, weights && !whole);
        if (weights && !whole) above = over_cluster(s, mine, 1, a.cluster, rank).all;
        else meet(a.cluster);
      }
      int n = s->have;        // entries of the list
      if (rank == 0) {
        n = r.join();
        // room for the sums, where this block's slice was
        u64* const sums = reinterpret_cast<u64*>(room);
        if (whole) {
          r.sum_up(sums);
          int kept = weights ? n : min(n, k);
          if (by_weight) {
            const u64 goal = weights ? target : p > 0.0f ? max(u64(1), fraction_of(sums[kept - 1], p, true)) : 1;
            const int unit = weights ? kCoarse : 0;
            kept = min(kept, count_of([&](int i) { return sums[i] >> unit < goal; }) + 1);
          }
          if (floor != kNoCut) kept = max(1, min(kept, count_of([&](int i) { return s->list[i] >= floor; })));
          draw_from_list(s, sums + kList, a, r.weigh, row, kept, sums[kept - 1], u);
        } else {
          int need = min(n, (int)(target - w.above));
          if (weights) {
            need = 1;
            if (target > above) {
              r.sum_up(s->weight);
              need = min(n, count_of([&](int i) { return s->weight[i] >> kCoarse < target - above; }) + 1);
            }
          }
          const u64 found = s->list[max(0, need - 1)];
          if (tid < a.cluster) remote_put(remote(&s->give[2], tid), found);
        }
      }
      if (whole) {
        drawn = true;
        break;
      }
      meet(a.cluster);
      cut = max(cut, s->give[2]);
      if (weights && floor <= cut) {
        // the kept tokens of the window, on top of those above it
        const u64 lowest = (u64)(kMaxVocab - (r.start + end)), highest = (u64)(kMaxVocab - 1 - (r.start + pad));
        for (int i = tid; i < n; i += kThreads) {
          const u64 q = s->list[i], at = q & kIndexMask;
          const float l = key_value((uint32_t)(q >> kIndexBits));
          if (q >= cut && at >= lowest && at <= highest && l >= r.weigh.least)
            atomicAdd(&s->sums[(kMaxVocab - 1 - (int)at - r.start) / kBlock], (u64)r.weigh.one(l));
        }
        summed = true;
      }
    }
    if (!drawn) {
      // ---- the kept weights by block, and the draw
      cut = max(cut, floor);
      const float lo = fmaxf(key_value(max((uint32_t)(cut >> kIndexBits), order_key(-INFINITY))), r.weigh.least);
      auto kept = [&](float l, int i) { return l >= lo && (l > lo || r.place(l, i) >= cut); };
      if (!summed) {
        u64 mine = 0;
        r.each([&](const float (&l)[4], int i) { mine += r.weigh_if(l, [&](int e) { return kept(l[e], i + e); }); },
               [&](int b) {
#pragma unroll
                 for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
                 if (lane == 0) s->sums[b] = mine;
                 mine = 0;
               });
      }
      __syncthreads();
      const int b0 = 2 * tid, b1 = b0 + 1;
      const u64 sum0 = b0 < r.blocks ? s->sums[b0] >> kCoarse : 0, sum1 = b1 < r.blocks ? s->sums[b1] >> kCoarse : 0;
      const Sum block = scan(s, sum0 + sum1);
      const Sum slices = over_cluster(s, block.all, 4, a.cluster, rank);
      const u64 goal = goal_of(slices.all, u);
      if (slices.before <= goal && goal < slices.before + block.all) {       // (the same for all threads of a block)
        const u64 at = slices.before + block.before;
        if (at <= goal && goal < at + sum0 + sum1) {
          const bool second = goal >= at + sum0;
          const int b = second ? b1 : b0;
          s->pick[0] = b;
          s->pick[1] = min((goal - at - (second ? sum0 : 0)) << kCoarse, s->sums[b] - 1);
        }
        __syncthreads();
        const int i = (int)s->pick[0] * kBlock + tid;
        const float l = r.value(i);
        const u64 mine = kept(l, i) ? r.weigh.one(l) : 0;
        const u64 before = scan(s, mine).before, place = s->pick[1];
        if (before <= place && place < before + mine)
          answer(a, r.weigh, row, r.start + i, l, slices.all, mine >> kCoarse == slices.all);
      }
    }
  }
  if (a.cluster > 1) meet(a.cluster);     // nothing of this block is read any more
}

template <typename T, bool kResident> cudaError_t launch_kernel(const Args& a, int64_t ntok, cudaStream_t s) {
  const auto kernel = sample_kernel<T, kResident>;
  const int slice = kResident ? (a.slice + kBlock) * (int)sizeof(T) : 0;
  const int smem = (int)sizeof(Shared) + std::max(slice, 2 * kList * (int)sizeof(u64));
  cudaError_t e = ensure_dynamic_smem((const void*)kernel, smem);
  if (e == cudaSuccess && a.cluster > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ntok * a.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T> cudaError_t launch_as(const SampleCall& c, cudaStream_t s) {
  Args a = {c.logits, c.stride, c.vocab, 0, 1, c.u, c.temperature, c.top_k, c.top_p, c.min_p, c.tokens, c.logp};
  // Thread blocks a row: as many as run at once (two an SM), where slices have
  // 2048 tokens at least.
  while (a.cluster < kMaxCluster && 2 * c.ntok * a.cluster <= kSlots && c.vocab > a.cluster * 2048) a.cluster *= 2;
  a.slice = ((c.vocab + a.cluster - 1) / a.cluster + 31) / 32 * 32;
  if (c.ntok * a.cluster > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // In shared memory where two slices fit into an SM's, else read again from L2.
  return a.slice * (int)sizeof(T) <= kMaxResident ? launch_kernel<T, true>(a, c.ntok, s)
                                                  : launch_kernel<T, false>(a, c.ntok, s);
}

}  // namespace

cudaError_t launch_sample(const SampleCall& c, cudaStream_t s) {
  switch (c.type) {
    case TQ_F32: return launch_as<float>(c, s);
    case TQ_F16: return launch_as<__half>(c, s);
    default: return launch_as<__nv_bfloat16>(c, s);
  }
}

}  // namespace tq
