// tq_sample.cu -- the draw of the next token: temperature, top-k, top-p, min-p
// and one given uniform number a row.
//
// The kept tokens are a beginning of the order (falling logit, rising index).
// A token's place in it is an integer, its logit's bits above its index, so
// each filter is a least integer, found by counting (top-k) or weighing (top-p)
// the tokens in 1024 ranges of it at a time.
#include <cmath>

#include "tq_requests.cuh"
#include "tq_weight.cuh"

namespace tq {
namespace {

constexpr int kThreads = 512;
constexpr int kBins = 1024;
constexpr int kIndexBits = 18;
static_assert(kMaxVocab == 1 << kIndexBits, "an index below a logit's bits");

__device__ const ExpTable g_exp_table = make_exp_table();

struct Args {
  const void* logits;
  int64_t stride;
  int vocab, vec;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logp;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ Args a) {
  __shared__ float2 table[kExpSteps];
  __shared__ unsigned long long bins[kBins];
  __shared__ float s_top[kThreads / 32];
  __shared__ int s_bad[kThreads / 32], s_at[kThreads / 32];
  __shared__ unsigned long long s_lo, s_hi, s_above;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, vocab = a.vocab;
  for (int j = tid; j < kExpSteps; j += kThreads) table[j] = g_exp_table.v[j];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const T* const x = static_cast<const T*>(a.logits) + row * a.stride;

  // the largest logit, its lowest index, and whether there is a NaN
  float top = -INFINITY;
  int at = 0x7fffffff, bad = 0;
  for (int i = tid; i < vocab; i += kThreads) {
    const float l = Elem<T>::up(x[i]);
    bad |= l != l;
    if (l > top) {
      top = l;
      at = i;
    }
  }
  for (int d = 16; d > 0; d >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, top, d);
    const int i = __shfl_xor_sync(0xffffffffu, at, d);
    if (t > top || (t == top && i < at)) {
      top = t;
      at = i;
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    s_top[warp] = top;
    s_at[warp] = at;
    s_bad[warp] = bad;
  }
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) {
    bad |= s_bad[w];
    if (s_top[w] > top || (s_top[w] == top && s_at[w] < at)) {
      top = s_top[w];
      at = s_at[w];
    }
  }
  const float temp = a.temperature ? a.temperature[row] : 1.0f;
  if (bad || top == -INFINITY || !(temp >= 0.0f) || temp == INFINITY) {
    if (tid == 0) {
      a.tokens[row] = -1;
      if (a.logp) a.logp[row] = NAN;
    }
    return;
  }
  if (temp < 0x1p-100f) {
    if (tid == 0) {
      a.tokens[row] = at;
      if (a.logp) a.logp[row] = 0.0f;
    }
    return;
  }
  const bool infinite = top == INFINITY;
  if (infinite) top = 0.0f;
  auto get = [&](int i) {
    const float l = Elem<T>::up(x[i]);
    return infinite ? (l == INFINITY ? 0.0f : -INFINITY) : l;
  };
  const double c = 1.4426950408889634074 / (double)temp;
  Weigher weigh;
  weigh.m = top;
  weigh.c_hi = (float)c;
  weigh.c_lo = (float)(c - (double)weigh.c_hi);
  weigh.table = table;
  auto place = [&](float l, int i) {
    return ((unsigned long long)order_key(l) << kIndexBits) | (unsigned)(kMaxVocab - 1 - i);
  };

  // The least place such that the tokens from it on (and from `from` on) number,
  // or weigh, `target` at least; they do from 0 on.
  auto find = [&](bool by_weight, unsigned long long target, unsigned long long from) {
    unsigned long long lo = 0, hi = (1ull << (32 + kIndexBits)) - 1, above = 0;
    for (int shift = 40; shift >= 0; shift -= 10) {
      for (int j = tid; j < kBins; j += kThreads) bins[j] = 0;
      __syncthreads();
      for (int i = tid; i < vocab; i += kThreads) {
        const float l = get(i);
        const unsigned long long q = place(l, i);
        if (q >= lo && q <= hi && q >= from)
          atomicAdd(&bins[(q - lo) >> shift], by_weight ? (unsigned long long)weigh(l) : 1ull);
      }
      __syncthreads();
      if (tid == 0) {
        int j = kBins - 1;
        for (; j > 0 && above + bins[j] < target; --j) above += bins[j];
        s_lo = lo + ((unsigned long long)j << shift);
        s_hi = s_lo + ((1ull << shift) - 1);
        s_above = above;
      }
      __syncthreads();
      lo = s_lo;
      hi = s_hi;
      above = s_above;
    }
    return lo;
  };

  unsigned long long cut = 0;
  const int k = a.top_k ? a.top_k[row] : 0;
  if (k > 0 && k < vocab) cut = find(false, k, 0);
  // sum of the weights from `cut` on, each thread a run of indexes
  const int run = (vocab + kThreads - 1) / kThreads, first = tid * run, last = min(vocab, first + run);
  __shared__ unsigned long long s_sum[kThreads];
  auto sum = [&]() {
    unsigned long long mine = 0;
    for (int i = first; i < last; ++i) {
      const float l = get(i);
      if (place(l, i) >= cut) mine += weigh(l);
    }
    __syncthreads();
    s_sum[tid] = mine;
    __syncthreads();
    unsigned long long all = 0;
    for (int j = 0; j < kThreads; ++j) all += s_sum[j];
    return all;
  };
  const float p = a.top_p ? a.top_p[row] : 1.0f;
  if (p < 1.0f) {
    const double want = ceil((double)p * (double)sum());
    cut = max(cut, find(true, want > 1.0 ? (unsigned long long)want : 1ull, cut));
  }
  const float mp = a.min_p ? a.min_p[row] : 0.0f;
  if (mp > 0.0f) {
    const float least = fminf(__double2float_ru((double)top + (double)temp * log((double)mp)), top);
    cut = max(cut, (unsigned long long)order_key(least) << kIndexBits);
  }
  const unsigned long long total = sum();
  const float u = a.u[row];
  unsigned long long target = u > 0.0f ? (unsigned long long)((double)u * (double)total) : 0;
  if (target >= total) target = total - 1;
  unsigned long long before = 0;
  for (int j = 0; j < tid; ++j) before += s_sum[j];
  if (before <= target && target < before + s_sum[tid]) {
    for (int i = first; i < last; ++i) {
      const float l = get(i);
      if (place(l, i) < cut) continue;
      before += weigh(l);
      if (before > target) {
        a.tokens[row] = i;
        if (a.logp)
          a.logp[row] = (float)(((double)l - (double)top) / (double)temp -
                                log((double)total * 0x1p-45));
        break;
      }
    }
  }
}

template <typename T> cudaError_t launch_as(const SampleCall& c, cudaStream_t s) {
  const Args a = {c.logits, c.stride, c.vocab, 0, c.u, c.temperature, c.top_k, c.top_p, c.min_p,
                  c.tokens, c.logp};
  return launch_pdl(sample_kernel<T>, dim3((unsigned)c.ntok), dim3(kThreads), 0, s, a);
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
