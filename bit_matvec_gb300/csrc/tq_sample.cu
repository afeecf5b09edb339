// tq_sample.cu -- the draw of the next token: temperature, top-k, top-p, min-p
// and one given uniform number a row.
//
// A cluster of thread blocks takes a row, each a slice of it that stays in its
// shared memory: logits are read from memory once, whatever the filters need.
//
// The kept tokens are a beginning of the order (falling logit, rising index). A
// token's place in it is an integer, its logit's bits above its complemented
// index, so each filter is a least place, the cut. A cut is found by counting
// (top-k) or weighing (top-p) the tokens in 1536 ranges, first 32 to an octave
// of weight, then, where a range holds too many tokens (equal logits), equal
// parts of it, until the range around the cut holds few enough to be sorted. If
// that range and all tokens above it fit in the list, which is the rule for the
// usual settings, everything else happens on the list. Otherwise a pass over the
// slices sums the kept weights in blocks of 512 tokens, and the block that the
// draw falls into is looked through.
//
// Weights are integers (tq_weight.cuh): their sums do not depend on the order
// in which threads add.
#include <algorithm>
#include <cmath>
#include <cstddef>

#include "tq_requests.cuh"
#include "tq_weight.cuh"

namespace tq {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kIndexBits = 18;
constexpr int kList = 1024;                 // tokens that are sorted
constexpr int kBlock = 512;                 // tokens of a sum
constexpr int kMaxSlice = 32768;            // tokens of a thread block: 2^15 times 2^16 fit in a bin
constexpr int kMaxBlocks = kMaxSlice / kBlock;
constexpr int kMaxCluster = 16;
static_assert(kMaxVocab == 1 << kIndexBits, "an index below a logit's bits");
static_assert(kBlock == kThreads, "a thread for each token of a block");
static_assert(kWeightBins % 4 == 0 && kWeightBins / 4 <= kThreads, "four bins a thread");

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
struct Shared {
  float2 table[kExpSteps];
  u64 list[kList];            // places of the tokens at a cut
  u64 weight[kList];          // (rank 0) their weights; while a window is narrowed, weights by bin
  uint32_t bins[kWeightBins]; // tokens, or leading bits of weights
  u64 sums[kMaxBlocks];       // kept weights by block
  u64 scan[kWarps];
  u64 give[4];                // what the other blocks of the cluster read
  int have;                   // entries of the list
  float top;
  int first;                  // lowest index of the largest logit
  u64 pick[6];
};

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

// floor(a * x) of a weight sum and a float in (0, 1), exactly; `up`: the ceiling.
__device__ __forceinline__ u64 fraction_of(u64 a, float x, bool up) {
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

template <typename T> struct Row {
  Shared& s;
  const T* const xs;          // this block's slice
  const Args& a;
  const int tid, lane, warp, rank, cluster;
  const int start, count, blocks;    // of the slice: its first token, tokens, blocks of 512
  Weigher weigh;

  // ---- the cluster and the block

  __device__ __forceinline__ void meet() const {
    if (cluster == 1) {
      __syncthreads();
      return;
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
  // The sum of the threads' values before this thread, and of all.
  __device__ __forceinline__ u64 scan(u64 v, u64& total) const {
    u64 sum = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const u64 o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    __syncthreads();      // (the last scan's readers are done)
    if (lane == 31) s.scan[warp] = sum;
    __syncthreads();
    u64 before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const u64 o = s.scan[w];
      if (w < warp) before += o;
      total += o;
    }
    return before + sum - v;
  }
  // The sum over the cluster of a value that all threads of a block have, by
  // way of give[at]; `before`: of the blocks before this one.
  __device__ __forceinline__ u64 over_cluster(u64 mine, int at, u64& before) const {
    if (tid == 0) s.give[at] = mine;
    meet();
    before = 0;
    u64 all = 0;
    for (int r = 0; r < cluster; ++r) {
      const u64 v = cluster == 1 ? mine : remote_u64(remote(&s.give[at], r));
      if (r < rank) before += v;
      all += v;
    }
    return all;
  }

  // ---- tokens

  __device__ __forceinline__ u64 place(float l, int i) const {   // i: within the slice
    return ((u64)order_key(l) << kIndexBits) | (unsigned)(kMaxVocab - 1 - (start + i));
  }
  // Calls f(logit, index within the slice) for every token, four of a thread at
  // a time; a warp's turn is a block of 512 tokens, after which `end(block)`.
  template <typename F, typename E> __device__ __forceinline__ void each(F f, E end) const {
    for (int b = warp; b < blocks; b += kWarps) {
      const int end_of = min(kBlock, count - b * kBlock);
#pragma unroll
      for (int j = 0; j < kBlock / 128; ++j) {
        const int o = j * 128 + lane * 4, i = b * kBlock + o;
        const Vec<T, 4> v = *reinterpret_cast<const Vec<T, 4>*>(xs + i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (o + e < end_of) f(Elem<T>::up(v.v[e]), i + e);
      }
      end(b);
    }
  }
  template <typename F> __device__ __forceinline__ void each(F f) const {
    each(f, [](int) {});
  }

  // ---- finding a cut

  struct Window {
    u64 lo, hi;       // places
    u64 above;        // by count: tokens above the window
    u64 inside;       // tokens in it, at most
  };

  // The least place of a weight's bin of at most b.
  __device__ __forceinline__ u64 bin_end(int b, uint32_t top_key) const {
    // the least key whose bin is at most b: 32 candidates a step
    uint32_t lo = 0, hi = top_key + 1;     // (above all tokens, if none has such a bin)
    while (lo < hi) {
      const uint32_t step = (hi - lo) / 32 + 1, at = lo + (uint32_t)lane * step;
      const bool in = at < hi && at >= lo && weigh.bin(key_value(at)) <= b;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (m) {
        const int l = __ffs(m) - 1;
        hi = lo + (uint32_t)l * step;
        if (l > 0) lo = lo + (uint32_t)(l - 1) * step + 1;
        else lo = hi;
      } else {
        const uint32_t l = min(31u, (hi - 1 - lo) / step);    // the last candidate below hi
        lo = lo + l * step + 1;
      }
    }
    return (u64)lo << kIndexBits;
  }

  // The range around the cut: by count, the least place such that `target`
  // tokens are at it or above; by weight, such that they weigh the share `share`
  // of all at least, whose sum goes to *all. Tokens from `from` on only.
  // Narrowed until at most kList tokens are inside.
  __device__ __forceinline__ Window search(bool by_weight, u64 target, u64 from, uint32_t top_key, u64* all,
                                           float share) {
    Window w = {from, ((u64)top_key << kIndexBits) | kIndexMask, 0, ~u64(0)};
    // (tokens that weigh nothing do not help to reach a weight)
    if (by_weight) w.lo = max(from, (u64)order_key(weigh.least) << kIndexBits);
    // ---- 32 ranges to an octave of weight
    meet();                              // (the last reading of the bins is over)
    for (int j = tid; j < kWeightBins; j += kThreads) s.bins[j] = 0;
    __syncthreads();
    u64 mine = 0;
    each([&](float l, int i) {
      if (from != kNoCut && place(l, i) < from) return;
      if (!by_weight) {
        atomicAdd(&s.bins[weigh.bin(l)], 1u);
      } else if (l >= weigh.least) {
        uint32_t top16;
        mine += weigh(l, &top16);
        atomicAdd(&s.bins[weigh.bin(l)], top16);
      }
    });
    u64 ignored;
    if (by_weight) {
      u64 sum;
      scan(mine, sum);
      *all = over_cluster(sum, 0, ignored);
      target = share > 0.0f ? max(u64(1), fraction_of(*all, share, true)) : 1;
    } else {
      meet();
    }
    // this thread's four bins, of all blocks: tokens (at most), and what counts, at least and at most
    u64 n[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0}, hi[4] = {0, 0, 0, 0};
    if (tid < kWeightBins / 4) {
      for (int r = 0; r < cluster; ++r) {
        const uint4 v = remote_u128(remote(&s.bins[4 * tid], r));
        n[0] += v.x;
        n[1] += v.y;
        n[2] += v.z;
        n[3] += v.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (by_weight) {
          // Sums of weights' first 16 bits, 2^15 - 8 at least (just below a
          // power of two the table's entry is that power's): a token for each of
          // these in the sum, at most, each cut by less than one and off by a unit.
          const int octave = (4 * tid + e + 31) / 32;
          const u64 tokens = (n[e] + (n[e] >> 11)) >> 15, v = (n[e] << 31) >> octave;
          lo[e] = v - min(v, tokens);
          hi[e] = tokens ? (((n[e] + tokens) << 31) >> octave) + tokens + 1 : 0;
          n[e] = tokens;
        } else {
          lo[e] = hi[e] = n[e];
        }
      }
    }
    pick_bins(n, lo, hi, target, 0);
    {
      const int first = (int)s.pick[0], last = (int)s.pick[1];
      const u64 low = last < kWeightBins ? bin_end(last, top_key) : 0;
      if (first > 0) w.hi = bin_end(first - 1, top_key) - 1;
      w.lo = max(w.lo, low);
      w.inside = s.pick[5] - s.pick[4];
      w.above = s.pick[2];
    }
    // ---- equal parts of the window, sums exact
    u64* const sums = s.list;
    static_assert(sizeof(s.list) + sizeof(s.weight) >= kWeightBins * sizeof(u64), "");
    static_assert(offsetof(Shared, weight) == offsetof(Shared, list) + sizeof(s.list), "one after the other");
    for (int level = 1; w.inside > kList; ++level) {
      int shift = 0;
      while (((w.hi - w.lo) >> shift) >= kWeightBins) ++shift;
      meet();
      for (int j = tid; j < kWeightBins; j += kThreads) {
        s.bins[j] = 0;
        sums[j] = 0;
      }
      __syncthreads();
      u64 above = 0;
      each([&](float l, int i) {
        const u64 q = place(l, i);
        const bool weighs = by_weight && l >= weigh.least;
        if (q > w.hi) {
          if (weighs) above += weigh(l);
        } else if (q >= w.lo) {
          const int j = (int)((w.hi - q) >> shift);
          atomicAdd(&s.bins[j], 1u);
          if (weighs) atomicAdd(&sums[j], (u64)weigh(l));
        }
      });
      if (by_weight) {
        u64 sum;
        scan(above, sum);
        w.above = over_cluster(sum, 0, ignored);
      } else {
        meet();
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) n[e] = lo[e] = 0;
      if (tid < kWeightBins / 4) {
        for (int r = 0; r < cluster; ++r) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            n[e] += remote_u32(remote(&s.bins[4 * tid + e], r));
            if (by_weight) lo[e] += remote_u64(remote(&sums[4 * tid + e], r));
          }
        }
      }
      pick_bins(n, by_weight ? lo : n, by_weight ? lo : n, target, w.above);
      const u64 end = w.hi, first = s.pick[0], last = s.pick[1];
      w.hi = end - (first << shift);
      w.lo = max(w.lo, end - min(end, ((last + 1) << shift) - 1));
      w.inside = s.pick[5] - s.pick[4];
      w.above = s.pick[2];
      if (w.inside <= kList) meet();     // (the last reading of the sums, where the list is, is over)
    }
    return w;
  }

  // Among the bins of all threads (n tokens at most; lo to hi of what counts, `above` before the
  // first): the first that may reach `target` in pick[0], what is before it in pick[2] and the tokens
  // in pick[4]; the first that surely does in pick[1] (kWeightBins if none), the tokens up to it in pick[5].
  __device__ __forceinline__ void pick_bins(const u64 (&n)[4], const u64 (&lo)[4], const u64 (&hi)[4], u64 target,
                                            u64 above) {
    u64 total, all_n;
    u64 at_lo = above + scan(lo[0] + lo[1] + lo[2] + lo[3], total);
    u64 at_hi = above + scan(hi[0] + hi[1] + hi[2] + hi[3], total);
    u64 at_n = scan(n[0] + n[1] + n[2] + n[3], all_n);
    if (tid == 0) {
      s.pick[0] = 0;
      s.pick[1] = kWeightBins;
      s.pick[2] = above;
      s.pick[4] = 0;
      s.pick[5] = all_n;
    }
    __syncthreads();
    if (tid < kWeightBins / 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (at_hi < target && at_hi + hi[e] >= target) {
          s.pick[0] = 4 * tid + e;
          s.pick[2] = at_lo;
          s.pick[4] = at_n;
        }
        if (at_lo < target && at_lo + lo[e] >= target) {
          s.pick[1] = 4 * tid + e;
          s.pick[5] = at_n + n[e];
        }
        at_lo += lo[e];
        at_hi += hi[e];
        at_n += n[e];
      }
    }
    __syncthreads();
  }

  // The tokens of the window in this block's list, and the weights of those
  // above it.
  __device__ __forceinline__ u64 gather(const Window& w, bool weights) {
    if (tid == 0) s.have = 0;
    __syncthreads();
    u64 above = 0;
    const float lo = key_value(max((uint32_t)(w.lo >> kIndexBits), order_key(-INFINITY)));
    each([&](float l, int i) {
      if (!(l >= lo)) return;
      const u64 q = place(l, i);
      if (q < w.lo) return;
      if (q > w.hi) {
        if (weights && l >= weigh.least) above += weigh(l);
        return;
      }
      const int at = atomicAdd(&s.have, 1);
      if (at < kList) s.list[at] = q;
    });
    u64 sum;
    scan(above, sum);
    return sum;
  }

  // (rank 0) All blocks' lists in this one's, sorted, the highest first; returns
  // their number. The weights are in s.weight.
  __device__ __forceinline__ int join() {
    int have[kMaxCluster], n = 0, mine = 0;
    if (cluster > 1) {
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) have[r] = r < cluster ? (int)remote_u32(remote(&s.have, r)) : 0;
      mine = have[0];
      u64 got[kList / kThreads];
#pragma unroll
      for (int j = 0; j < kList / kThreads; ++j) {
        const int want = mine + j * kThreads + tid;
        int at = want - mine;
        got[j] = 0;
        bool done = false;
#pragma unroll
        for (int r = 1; r < kMaxCluster; ++r) {
          if (!done && at < have[r]) {
            got[j] = remote_u64(remote(&s.list[at], r));
            done = true;
          }
          if (!done) at -= have[r];
        }
        if (want < kList) s.list[want] = got[j];
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) n += have[r];
    } else {
      __syncthreads();
      n = mine = s.have;
      for (int i = mine + tid; i < kList; i += kThreads) s.list[i] = 0;
    }
    n = min(n, kList);
    __syncthreads();
    sort(s.list, n);
    for (int i = tid; i < kList; i += kThreads) {
      const float l = key_value((uint32_t)(s.list[i] >> kIndexBits));
      s.weight[i] = i < n && l >= weigh.least ? weigh(l) : 0;
    }
    __syncthreads();
    return n;
  }
  // The first n of kList values, falling; what lies behind them is 0 up to the
  // next power of two.
  __device__ __forceinline__ void sort(u64* v, int n) const {
    int size = 2;
    while (size < n) size *= 2;
    for (int k = 2; k <= size; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int i = tid; i < size / 2; i += kThreads) {
          const int a = 2 * i - (i & (j - 1)), b = a + j;
          const u64 x = v[a], y = v[b];
          if ((x < y) == ((a & k) == 0)) {
            v[a] = y;
            v[b] = x;
          }
        }
        __syncthreads();
      }
  }
  // (rank 0) The number of sorted entries, at least 1, that are needed for the
  // weights to sum to `target`; `before`: the weights before each thread's two.
  __device__ __forceinline__ int needed(int n, u64 target) {
    static_assert(kList == 2 * kThreads, "two entries a thread");
    const u64 x = s.weight[2 * tid], y = s.weight[2 * tid + 1];
    u64 total;
    const u64 at = scan(x + y, total);
    const int less = (at + x < target ? 1 : 0) + (at + x + y < target ? 1 : 0);
    u64 all;
    scan((u64)less, all);
    return max(1, min(n, (int)all + 1));
  }
  // (rank 0) The sum of the first n entries' weights.
  __device__ __forceinline__ u64 weight_of(int n) {
    u64 total;
    scan((2 * tid < n ? s.weight[2 * tid] : 0) + (2 * tid + 1 < n ? s.weight[2 * tid + 1] : 0), total);
    return total;
  }

  __device__ __forceinline__ void answer(int64_t row, int token, float l, double temp, u64 total) const {
    a.tokens[row] = token;
    if (!a.logp) return;
    // ln(w / total) = l / T - R ln 2 - ln(total / 2^46)
    const double c = 1.4426950408889634074 / temp, r = 6144.0 - (double)weigh.k;
    const double e = weigh.far ? ((double)l - (double)weigh.m) * c : (double)l * c;
    a.logp[row] = (float)((e - r) * 0.69314718055994530942 - log((double)total * 0x1p-46));
  }

  // (rank 0) The draw from a sorted list that holds all kept tokens.
  __device__ __forceinline__ void draw_from_list(int64_t row, int kept, double temp, float u) {
    const u64 total = weight_of(kept);
    const u64 goal = u > 0.0f ? (u < 1.0f ? min(fraction_of(total, u, false), total - 1) : total - 1) : 0;
    // by rising index: the complemented index, then the entry
    u64 again[kList / kThreads];
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) {
      const int i = tid + j * kThreads;
      again[j] = i < kept ? u64(1) << 63 | (s.list[i] & kIndexMask) << 10 | (u64)i : 0;
    }
    static_assert(kList == 1 << 10, "an entry below an index");
    __syncthreads();
    u64* const by_index = reinterpret_cast<u64*>(s.table);     // (the weights are all computed)
    static_assert(sizeof(s.table) >= kList * sizeof(u64), "");
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) by_index[tid + j * kThreads] = again[j];
    __syncthreads();
    sort(by_index, kept);
    const u64 p = by_index[2 * tid], q = by_index[2 * tid + 1];
    const u64 x = p ? s.weight[p & (kList - 1)] : 0, y = q ? s.weight[q & (kList - 1)] : 0;
    u64 sum;
    const u64 at = scan(x + y, sum);
    if (at <= goal && goal < at + x + y) {
      const int i = (int)((goal < at + x ? p : q) & (kList - 1));
      const u64 e = s.list[i];
      answer(row, kMaxVocab - 1 - (int)(e & kIndexMask), key_value((uint32_t)(e >> kIndexBits)), temp, total);
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  T* const xs = reinterpret_cast<T*>(raw + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  const int64_t row = blockIdx.x / a.cluster;
  const int start = rank * a.slice, count = max(0, min(a.slice, a.vocab - start));
  const int blocks = (count + kBlock - 1) / kBlock;
  for (int j = tid; j < kExpSteps; j += kThreads) s.table[j] = g_exp_table.v[j];
  if (tid == 0) s.first = 0x7fffffff;
  pdl_wait_primary();
  pdl_launch_dependents();
  Row<T> r = {s, xs, a, tid, lane, warp, rank, a.cluster, start, count, blocks, {}};

  // ---- the slice, its largest logit, and whether there is a NaN
  const float temp = a.temperature ? a.temperature[row] : 1.0f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.0f, mp = a.min_p ? a.min_p[row] : 0.0f, u = a.u[row];
  const T* const x = static_cast<const T*>(a.logits) + row * a.stride + start;
  float top = -INFINITY;
  {
    constexpr int kPiece = 16 / (int)sizeof(T);
    const int pieces = (uintptr_t)x % 16 == 0 ? count / kPiece : 0;
#pragma unroll 4
    for (int i = tid; i < pieces; i += kThreads) {
      const uint4 q = ldg_stream_v4(reinterpret_cast<const uint4*>(x) + i);
      reinterpret_cast<uint4*>(xs)[i] = q;
      const Vec<T, kPiece> v = *reinterpret_cast<const Vec<T, kPiece>*>(&q);
#pragma unroll
      for (int e = 0; e < kPiece; ++e) top = max_or_nan(top, Elem<T>::up(v.v[e]));
    }
#pragma unroll 8
    for (int i = pieces * kPiece + tid; i < count; i += kThreads) {
      const T v = x[i];
      xs[i] = v;
      top = max_or_nan(top, Elem<T>::up(v));
    }
    for (int i = count + tid; i < blocks * kBlock; i += kThreads) xs[i] = Elem<T>::down(-INFINITY);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
  float* const tops = reinterpret_cast<float*>(s.scan);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = max_or_nan(top, tops[w]);
  if (a.cluster > 1) {
    if (tid == 0) s.top = top;
    r.meet();
    for (int c = 0; c < a.cluster; ++c) top = max_or_nan(top, __uint_as_float(remote_u32(remote(&s.top, c))));
  }
  const bool none = top != top || top == -INFINITY || !(temp >= 0.0f) || temp == INFINITY;
  if (none) {
    if (rank == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.logp) a.logp[row] = NAN;
    }
  } else if (temp < 0x1p-100f) {
    int first = 0x7fffffff;
    r.each([&](float l, int i) {
      if (l == top) first = min(first, start + i);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) atomicMin(&s.first, first);
    r.meet();
    if (rank == 0 && tid == 0) {
      first = s.first;
      for (int c = 1; c < a.cluster; ++c) first = min(first, (int)remote_u32(remote(&s.first, c)));
      a.tokens[row] = first;
      if (a.logp) a.logp[row] = 0.0f;
    }
  } else {
    if (top == INFINITY) {
      // beside it every other logit is minus infinity
      for (int i = tid; i < blocks * kBlock; i += kThreads)
        xs[i] = Elem<T>::down(Elem<T>::up(xs[i]) == INFINITY ? 0.0f : -INFINITY);
      top = 0.0f;
      __syncthreads();
    }
    const double t = fmin((double)temp, 0x1p100);
    r.weigh.set(top, (float)t, s.table);
    const uint32_t top_key = order_key(top);
    u64 floor = kNoCut;       // of min-p
    if (mp > 0.0f) {
      const float least = fminf(__double2float_ru((double)top + t * log((double)mp)), top);
      floor = (u64)order_key(least) << kIndexBits;
    }
    const bool by_count = k > 0 && k < a.vocab, by_weight = p < 1.0f;
    // 0: not decided, 1: the list holds all kept tokens (rank 0 draws), 2: a cut
    bool drawn = false;
    u64 cut = kNoCut;
    for (int which = 0; which < 2 && !drawn; ++which) {
      if (which == 0 ? !by_count : !by_weight) continue;
      u64 target = (u64)k, sum = 0, before;
      const auto w = r.search(which == 1, target, cut, top_key, which == 1 ? &sum : nullptr, p);
      if (which == 1) target = p > 0.0f ? max(u64(1), fraction_of(sum, p, true)) : 1;
      // top-k with all tokens above it in the list: nothing else is kept
      const bool whole = which == 0 && w.above + w.inside <= kList;
      const auto range = whole ? typename Row<T>::Window{w.lo, ((u64)top_key << kIndexBits) | kIndexMask, 0, 0} : w;
      const u64 mine = r.gather(range, which == 1);
      const u64 above = r.over_cluster(mine, 1, before);
      if (rank == 0) {
        const int n = r.join();
        if (whole) {
          int kept = min(n, k);
          if (by_weight) {
            const u64 goal = p > 0.0f ? max(u64(1), fraction_of(r.weight_of(kept), p, true)) : 1;
            kept = min(kept, r.needed(kept, goal));
          }
          if (floor != kNoCut) {
            u64 over;
            r.scan((2 * tid < kept && s.list[2 * tid] >= floor ? 1 : 0) +
                       (2 * tid + 1 < kept && s.list[2 * tid + 1] >= floor ? 1 : 0), over);
            kept = max(1, (int)over);
          }
          r.draw_from_list(row, kept, t, u);
        } else {
          const int need = which == 0 ? min(n, (int)(target - w.above)) : target > above ? r.needed(n, target - above) : 1;
          const u64 found = s.list[max(0, need - 1)];
          if (tid < a.cluster) remote_put(remote(&s.give[2], tid), found);
        }
      }
      if (whole) {
        drawn = true;
      } else {
        r.meet();
        cut = max(cut, s.give[2]);
      }
    }
    if (!drawn) {
      cut = max(cut, floor);
      // ---- the kept weights by block, and the draw
      const float lo = cut == kNoCut ? r.weigh.least : fmaxf(key_value((uint32_t)(cut >> kIndexBits)), r.weigh.least);
      u64 mine = 0;
      r.each([&](float l, int i) {
        if (l >= lo && (cut == kNoCut || r.place(l, i) >= cut)) mine += r.weigh(l);
      }, [&](int b) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
        if (lane == 0) s.sums[b] = mine;
        mine = 0;
      });
      __syncthreads();
      u64 sum, before;
      const u64 to_block = r.scan(tid < blocks ? s.sums[tid] : 0, sum);
      const u64 total = r.over_cluster(sum, 3, before);
      const u64 goal = u > 0.0f ? (u < 1.0f ? min(fraction_of(total, u, false), total - 1) : total - 1) : 0;
      if (before <= goal && goal < before + sum) {       // (the same for all threads of a block)
        const u64 at = before + to_block;
        if (tid < blocks && at <= goal && goal < at + s.sums[tid]) {
          s.pick[0] = tid;
          s.pick[1] = at;
        }
        __syncthreads();
        const int i = (int)s.pick[0] * kBlock + tid;
        const u64 base = s.pick[1];
        const float l = Elem<T>::up(xs[i]);
        const u64 mine = l >= lo && (cut == kNoCut || r.place(l, i) >= cut) ? r.weigh(l) : 0;
        u64 all;
        const u64 from = base + r.scan(mine, all);
        if (from <= goal && goal < from + mine) r.answer(row, start + i, l, t, total);
      }
    }
  }
  if (a.cluster > 1) r.meet();     // nothing of this block is read any more
}

template <typename T> cudaError_t launch_as(const SampleCall& c, cudaStream_t s) {
  Args a = {c.logits, c.stride, c.vocab, 0, 1, c.u, c.temperature, c.top_k, c.top_p, c.min_p, c.tokens, c.logp};
  // Thread blocks a row: slices of at most 64 KB, two blocks an SM; more while
  // SMs are free and slices have 2048 tokens.
  constexpr int kSlice = std::min(kMaxSlice, 65536 / (int)sizeof(T));
  while (a.cluster < kMaxCluster &&
         (c.vocab > a.cluster * kSlice || (c.ntok * a.cluster < 152 && c.vocab > a.cluster * 2048)))
    a.cluster *= 2;
  a.slice = ((c.vocab + a.cluster - 1) / a.cluster + kBlock - 1) / kBlock * kBlock;
  if (c.ntok * a.cluster > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const auto kernel = sample_kernel<T>;
  const int smem = (int)sizeof(Shared) + a.slice * (int)sizeof(T);
  cudaError_t e = ensure_dynamic_smem((const void*)kernel, smem);
  if (e == cudaSuccess && a.cluster > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(c.ntok * a.cluster));
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

}  // namespace

cudaError_t launch_sample(const SampleCall& c, cudaStream_t s) {
  switch (c.type) {
    case TQ_F32: return launch_as<float>(c, s);
    case TQ_F16: return launch_as<__half>(c, s);
    default: return launch_as<__nv_bfloat16>(c, s);
  }
}

}  // namespace tq
