// tq_attn_api.cu -- the C ABI of the norm/rotation, append and attention
// calls: argument checks, planning, error reporting.
#include <algorithm>
#include <climits>
#include <cmath>

#include "tq_attn.cuh"

namespace tq {
namespace {

bool type_ok(int t) { return t == TQ_F32 || t == TQ_F16 || t == TQ_BF16; }
int64_t type_bytes(int t) { return t == TQ_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0; }

constexpr int64_t kMaxSize = int64_t(1) << 40;   // of a stride
bool size_ok(int64_t n) { return n >= 0 && n <= kMaxSize; }

// Whether n rows `stride` apart (both not negative) span at most 2^58 values:
// no memory holds more, and sums of such products stay in 64 bits.
bool span_ok(int64_t n, int64_t stride) { return n <= 1 || stride <= (int64_t(1) << 58) / (n - 1); }

int fail_cuda(cudaError_t e) {
  record_cuda_error(e);
  return TQ_ERR_CUDA;
}

struct Range {
  const char* p;
  int64_t n;
};
Range range(const void* p, int64_t n) { return {static_cast<const char*>(p), p ? n : 0}; }
bool overlap(Range a, Range b) {
  return a.n > 0 && b.n > 0 && a.p < b.p + b.n && b.p < a.p + a.n;
}

// Bytes from the first to the last value of [n][heads][dim] with token stride.
int64_t rows_bytes(int64_t n, int64_t stride, int64_t heads, int64_t dim, int type) {
  return n <= 0 || heads <= 0 ? 0 : ((n - 1) * stride + heads * dim) * type_bytes(type);
}

// Two buffers whose rows are interleaved in one projection (the same stride,
// both rows within it) overlap only where the rows do.
bool rows_overlap(const void* a, int64_t a_stride, int64_t a_row, int a_type, const void* b,
                  int64_t b_stride, int64_t b_row, int b_type, int64_t n) {
  if (n <= 0 || a_row <= 0 || b_row <= 0) return false;
  const int64_t as = a_stride * type_bytes(a_type), bs = b_stride * type_bytes(b_type);
  const int64_t ar = a_row * type_bytes(a_type), br = b_row * type_bytes(b_type);
  if (!overlap(range(a, (n - 1) * as + ar), range(b, (n - 1) * bs + br))) return false;
  if (as != bs || n == 1) return true;
  // the distance from a's rows to b's, within one stride
  int64_t d = ((intptr_t)b - (intptr_t)a) % as;
  if (d < 0) d += as;
  return d < ar || d + br > as;
}

int64_t cache_bytes(const tq_paged_kv& c) {
  if (c.pages <= 0 || c.heads <= 0) return 0;
  return ((c.pages - 1) * c.page_stride + (c.heads - 1) * c.head_stride +
          (c.page_size - 1) * c.slot_stride + c.head_dim) * 2;
}

int check_cache(const tq_paged_kv* c) {
  if (!c) return TQ_ERR_NULL;
  if (c->nseq < 0 || c->nseq > kMaxPositions || c->table_width < 0 || c->table_width > 0x7fffffff ||
      !size_ok(c->table_stride) || c->table_stride < c->table_width || c->pages < 1 ||
      c->pages > 0x7ffffffe || c->page_size < 8 || c->page_size % 8 != 0 ||
      c->page_size > (1 << 24) || c->heads < 1 || c->heads > 65535 || c->head_dim < 8 ||
      c->head_dim % 8 != 0 || c->head_dim > kMaxKvDim)
    return TQ_ERR_SHAPE;
  for (int64_t s : {c->page_stride, c->head_stride, c->slot_stride})
    if (s < 0 || s >= (int64_t(1) << 39) || s % 8 != 0) return TQ_ERR_SHAPE;
  if (!span_ok(c->nseq, c->table_stride) || !span_ok(c->pages, c->page_stride) ||
      !span_ok(c->heads, c->head_stride) || !span_ok(c->page_size, c->slot_stride))
    return TQ_ERR_SHAPE;
  if (c->slot_stride < c->head_dim || (c->heads > 1 && c->head_stride < c->head_dim) ||
      (c->pages > 1 && c->page_stride < c->head_dim))
    return TQ_ERR_SHAPE;
  if (c->type != TQ_F16 && c->type != TQ_BF16) return TQ_ERR_TYPE;
  return TQ_OK;
}

// The pointers of a cache that is going to be used.
int check_cache_pointers(const tq_paged_kv& c) {
  if (!c.k || !c.v || !c.block_table) return TQ_ERR_NULL;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.block_table, 4)) return TQ_ERR_ALIGN;
  return TQ_OK;
}

// Rotation, weights and positions shared by the two calls; fills `c`.
int take_rope(RopeCall& c, const float* qw, const float* kw, float eps, const tq_rope* rope,
              const int32_t* positions, int64_t head_dim, bool need_positions) {
  if (!(eps >= 0) || !std::isfinite(eps)) return TQ_ERR_SHAPE;
  c.head_dim = (int)head_dim;
  c.eps = eps;
  c.amplitude = 1.0f;
  if (rope && rope->rot_dim != 0) {
    if (rope->rot_dim < 0 || rope->rot_dim % 2 != 0 || rope->rot_dim > head_dim ||
        !std::isfinite(rope->amplitude))
      return TQ_ERR_SHAPE;
    if (!rope->turns) return TQ_ERR_NULL;
    if (!aligned(rope->turns, 8)) return TQ_ERR_ALIGN;
    c.half = (int)(rope->rot_dim / 2);
    c.interleaved = rope->interleaved != 0;
    c.amplitude = rope->amplitude;
    c.turns = rope->turns;
    need_positions = true;
  }
  if (need_positions && !positions) return TQ_ERR_NULL;
  if (!aligned(positions, 4) || !aligned(qw, 4) || !aligned(kw, 4)) return TQ_ERR_ALIGN;
  c.positions = positions;
  return TQ_OK;
}

// The planner's idea of the GPU.
constexpr int64_t kPlanSms = 152;
constexpr int64_t kCutBytes = 32;   // a CutTile of the kernel for many rows

// Limit of rows of a head and of positions, so that sums of two stay in 32 bits.
static_assert(kMaxPositions <= (1 << 30), "32-bit arithmetic of the kernels");

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

AttnPlan attn_plan(int64_t nseq, int64_t ntok, int64_t q_heads, int64_t kv_heads,
                   int64_t head_dim, int64_t max_q, int64_t max_kv, int64_t window) {
  AttnPlan p = {};
  const int64_t group = q_heads / kv_heads;
  if (max_q > ntok) max_q = ntok;
  if (window >= kMaxPositions) window = 0;   // as long as any sequence: none, as for the kernels
  const int64_t rows = max_q * group;
  // keys that the tokens of `n` rows see at most
  auto span_of = [&](int64_t n) {
    const int64_t s = window + std::min(max_q, n / group + 2);
    return window > 0 && s < max_kv ? s : max_kv;
  };

  // The kernel for few rows: 16, 32 or 64 of them a block, and the split of the
  // keys with the least time, in ns: rounds of blocks, each the key tiles of
  // one range (measured 0.5, 0.8 and 1.8 us a tile) and what starting and
  // ending a block takes (2 us, 5 with 64 rows), blocks of sequences too short
  // for their row tile, and the join. One round where blocks are few, several
  // short ones (which ragged lengths fill better) where they are many. A
  // cluster joins the ranges of a row tile where all blocks run at once; over
  // several rounds its blocks would hold their places until the longest ends
  // (239 us instead of 207 for 64 ragged sequences of up to 8192 positions),
  // and larger clusters do not fill every last place (40 clusters of 7 took two
  // rounds: 27 us, where 40 of 6 take 18).
  p.tile_rows = rows > 32 ? 64 : rows > 16 ? 32 : 16;
  p.key_tile = head_dim <= 64 ? 128 : 64;
  p.tiles_x = std::max<int64_t>(ceil_div(rows, p.tile_rows), 1);
  const int64_t slots = 2 * kPlanSms;
  const double blocks = (double)(kv_heads * nseq) * p.tiles_x;   // the largest sizes pass 64 bits
  // row tiles of `n` rows that there can be; the rest of the blocks end at once
  auto row_tiles_of = [&](int64_t n) {
    return kv_heads * std::min((double)nseq * ceil_div(rows, n), (double)(ntok * group / n) + nseq);
  };
  const bool wide = p.tile_rows == 64;
  const double units = row_tiles_of(p.tile_rows);
  const int64_t span = span_of(p.tile_rows);
  // in tiles, one more where the window does not start on one
  const int64_t tiles = std::max<int64_t>(ceil_div(span, p.key_tile) + (span < max_kv ? 1 : 0), 1);
  const int64_t tile_ns = wide ? 1800 : p.tile_rows == 32 ? 800 : 500;
  auto clustered = [&](int64_t s) {
    return s <= kMaxCluster && blocks * s <= (s <= 2 ? slots : slots * 17 / 20);
  };
  int64_t split = 1;
  double few_ns = INFINITY;
  for (int64_t s = 1; s <= tiles && s <= kMaxSplits; ++s) {
    const int64_t join = s == 1 ? 0 : clustered(s) ? 1000 : 3500;
    const double full = units * s / slots, up = std::ceil(full);
    const double rounds = wide && full > 1 ? (full + up) / 2 : up;
    const double ns = rounds * (ceil_div(tiles, s) * tile_ns + (wide ? 5000 : 2000)) + join + 2000 +
                      (blocks - units) * s / slots * 1500;
    if (ns < few_ns) {
      few_ns = ns;
      split = s;
    }
    if (blocks * s > (wide ? 2 : 16) * slots) break;
  }

  // The kernel for many rows: its start, end and join (more than 128 rows: twice
  // the partial results), the key tiles of 256 rows (128 rows: alternate ones)
  // dealt evenly to the SMs, and row tiles beyond one an SM. With 16 rows the
  // other is as fast as the memory in any case. Both measured, heads of 128,
  // few-row kernel first: 64 rows of one sequence over 9001 positions 19 and 23
  // us, 128 rows 25 and 25, 256 rows 39 and 32; 128 rows of 16 ragged sequences
  // 163 and 89; 274 tokens of 8 heads on one over 521 positions 12 and 24; 8
  // ragged sequences of 16 heads on 4 and up to 1000 positions, 64 new tokens
  // 23 and 30, 200 new tokens 42 and 39; 200 single tokens and 2 x 16 over up to
  // 500 positions 49 and 82. Of 105 shapes around the border, heads of 80 and 128
  // lose at most 3.4% to the other kernel, heads of 64, whose times these are not,
  // 27% and 13% in two of 35 (8 ragged sequences of 200 new tokens, 32 heads on
  // 4, up to 1000 positions: 46 us where the few-row kernel takes 36).
  const double row_tiles = row_tiles_of(256);
  const double many_ns = 18500 + (rows > 128 ? 7500 : 0) +
                         row_tiles * ceil_div(span_of(256), 128) * (rows > 128 ? 1600 : 1300) / kPlanSms +
                         std::max(row_tiles / kPlanSms - 1, 0.0) * 8000;
  if (rows > 16 && many_ns < few_ns) {
    p.chunk = true;
    p.tile_rows = 256;
    p.key_tile = 128;
    p.tiles_x = ntok * group / p.tile_rows + nseq;
    p.blocks = (int)kPlanSms;
    p.nsplit = p.cluster = 1;
    p.part_rows = 2 * kPlanSms * p.tile_rows;
    p.ws_bytes = ceil_div(p.part_rows * (head_dim + 1) * 4, 16) * 16 + kPlanSms * kCutBytes;
    return p;
  }
  p.chunk_tiles = (int)ceil_div(tiles, split);
  p.nsplit = (int)ceil_div(tiles, p.chunk_tiles);
  p.cluster = clustered(p.nsplit) ? p.nsplit : 1;
  p.part_rows = p.nsplit > p.cluster ? p.nsplit * ntok * q_heads : 0;
  p.ws_bytes = ceil_div(p.part_rows * (head_dim + 1) * 4, 16) * 16;
  return p;
}

}  // namespace tq

using namespace tq;

extern "C" {

int tq_qk_norm_rope(const void* Xq, int64_t xq_stride, const void* Xk, int64_t xk_stride,
                    int x_type, void* Yq, int64_t yq_stride, void* Yk, int64_t yk_stride,
                    int y_type, int64_t ntok, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                    const float* q_weight, const float* k_weight, float eps, const tq_rope* rope,
                    const int32_t* positions, void* stream) {
  if (ntok < 0 || ntok > 0x7fffffff || q_heads < 0 || k_heads < 0 || q_heads > 65535 ||
      k_heads > 65535 || head_dim < 2 || head_dim % 2 != 0 || head_dim > kMaxRopeDim)
    return TQ_ERR_SHAPE;
  for (int64_t s : {xq_stride, xk_stride, yq_stride, yk_stride})
    if (!size_ok(s) || !span_ok(ntok, s)) return TQ_ERR_SHAPE;
  if (!type_ok(x_type) || !type_ok(y_type)) return TQ_ERR_TYPE;
  if (ntok == 0 || q_heads + k_heads == 0) return TQ_OK;
  RopeCall c = {};
  const struct {
    const void* x;
    void* y;
    int64_t xs, ys, heads;
    const float* w;
  } in[2] = {{Xq, Yq, xq_stride, yq_stride, q_heads, q_weight},
             {Xk, Yk, xk_stride, yk_stride, k_heads, k_weight}};
  for (int k = 0; k < 2; ++k) {
    if (!in[k].heads) continue;
    const int64_t row = in[k].heads * head_dim;
    if (ntok > 1 && (in[k].xs < row || in[k].ys < row)) return TQ_ERR_SHAPE;
    if (!in[k].x || !in[k].y) return TQ_ERR_NULL;
    if (!aligned(in[k].x, type_bytes(x_type)) || !aligned(in[k].y, type_bytes(y_type)))
      return TQ_ERR_ALIGN;
    c.set[k] = {in[k].x, in[k].y, in[k].w, in[k].xs, in[k].ys, (int)in[k].heads, 1};
  }
  int rc = take_rope(c, q_weight, k_weight, eps, rope, positions, head_dim, false);
  if (rc != TQ_OK) return rc;
  for (int k = 0; k < 2; ++k) {
    const int64_t row = in[k].heads * head_dim;
    for (int j = 0; j < 2; ++j) {
      const int64_t other = in[j].heads * head_dim;
      const bool same = in[k].y == in[j].x && in[k].ys == in[j].xs && x_type == y_type && k == j;
      if (!same && rows_overlap(in[k].y, in[k].ys, row, y_type, in[j].x, in[j].xs, other, x_type, ntok))
        return TQ_ERR_ALIAS;
    }
    const Range y = range(in[k].y, rows_bytes(ntok, in[k].ys, in[k].heads, head_dim, y_type));
    if (overlap(y, range(q_weight, head_dim * 4)) || overlap(y, range(k_weight, head_dim * 4)) ||
        overlap(y, range(c.turns, c.half * 8)) || overlap(y, range(c.positions, ntok * 4)))
      return TQ_ERR_ALIAS;
  }
  if (rows_overlap(Yq, yq_stride, q_heads * head_dim, y_type, Yk, yk_stride, k_heads * head_dim,
                   y_type, ntok))
    return TQ_ERR_ALIAS;
  c.x_type = x_type;
  c.y_type = y_type;
  c.ntok = ntok;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  note_other_kernel(s);
  const cudaError_t e = launch_norm_rope(c, s);
  return e == cudaSuccess ? TQ_OK : fail_cuda(e);
}

int tq_kv_append(const void* Xq, int64_t xq_stride, const void* Xk, int64_t xk_stride,
                 const void* Xv, int64_t xv_stride, int x_type, void* Yq, int64_t yq_stride,
                 const tq_paged_kv* kv, const int32_t* seq_ids, const int32_t* positions,
                 int64_t ntok, int64_t q_heads, const float* q_weight, const float* k_weight,
                 float eps, const tq_rope* rope, void* stream) {
  int rc = check_cache(kv);
  if (rc != TQ_OK) return rc;
  if (ntok < 0 || ntok > 0x7fffffff || q_heads < 0 || q_heads > 65535) return TQ_ERR_SHAPE;
  for (int64_t s : {xq_stride, xk_stride, xv_stride, yq_stride})
    if (!size_ok(s) || !span_ok(ntok, s)) return TQ_ERR_SHAPE;
  if (!type_ok(x_type)) return TQ_ERR_TYPE;
  if (ntok == 0) return TQ_OK;
  const int64_t dim = kv->head_dim, xb = type_bytes(x_type);
  const int64_t q_row = q_heads * dim, kv_row = kv->heads * dim;
  if (ntok > 1 && (xk_stride < kv_row || xv_stride < kv_row || xq_stride < q_row || yq_stride < q_row))
    return TQ_ERR_SHAPE;
  if (!Xk || !Xv || !seq_ids || !positions || (q_heads && (!Xq || !Yq))) return TQ_ERR_NULL;
  rc = check_cache_pointers(*kv);
  if (rc != TQ_OK) return rc;
  if (!aligned(Xk, xb) || !aligned(Xv, xb) || !aligned(seq_ids, 4) ||
      (q_heads && (!aligned(Xq, xb) || !aligned(Yq, 2))))
    return TQ_ERR_ALIGN;
  RopeCall c = {};
  rc = take_rope(c, q_weight, k_weight, eps, rope, positions, dim, true);
  if (rc != TQ_OK) return rc;
  // what is written: the two caches and Yq
  const Range in[] = {range(q_heads ? Xq : nullptr, rows_bytes(ntok, xq_stride, q_heads, dim, x_type)),
                      range(Xk, rows_bytes(ntok, xk_stride, kv->heads, dim, x_type)),
                      range(Xv, rows_bytes(ntok, xv_stride, kv->heads, dim, x_type)),
                      range(seq_ids, ntok * 4), range(positions, ntok * 4),
                      range(q_weight, dim * 4), range(k_weight, dim * 4), range(c.turns, c.half * 8),
                      range(kv->block_table,
                            kv->nseq > 0 ? ((kv->nseq - 1) * kv->table_stride + kv->table_width) * 4 : 0)};
  const Range out[] = {range(kv->k, cache_bytes(*kv)), range(kv->v, cache_bytes(*kv)),
                       range(q_heads ? Yq : nullptr, rows_bytes(ntok, yq_stride, q_heads, dim, kv->type))};
  for (int i = 0; i < 3; ++i)
    for (const Range& r : in) {
      if (!overlap(out[i], r)) continue;
      // Yq beside the inputs in one strided buffer, or over Xq itself
      const bool x = i == 2 && r.n > 0 && kv->type == x_type && yq_stride == xq_stride;
      if (x && Yq == Xq && &r == &in[0]) continue;
      if (x && xk_stride == yq_stride && &r == &in[1] &&
          !rows_overlap(Yq, yq_stride, q_row, x_type, Xk, xk_stride, kv_row, x_type, ntok))
        continue;
      if (x && xv_stride == yq_stride && &r == &in[2] &&
          !rows_overlap(Yq, yq_stride, q_row, x_type, Xv, xv_stride, kv_row, x_type, ntok))
        continue;
      return TQ_ERR_ALIAS;
    }
  // keys and values interleaved in one allocation are a choice of strides; the
  // same start is not
  if (kv->k == kv->v || overlap(out[0], out[2]) || overlap(out[1], out[2])) return TQ_ERR_ALIAS;
  if (q_heads) c.set[0] = {Xq, Yq, q_weight, xq_stride, yq_stride, (int)q_heads, 1};
  c.set[1] = {Xk, nullptr, k_weight, xk_stride, 0, (int)kv->heads, 1};
  c.set[2] = {Xv, nullptr, nullptr, xv_stride, 0, (int)kv->heads, 0};
  c.x_type = x_type;
  c.y_type = kv->type;
  c.ntok = ntok;
  c.append = 1;
  c.seq_ids = seq_ids;
  c.kv = *kv;
  cudaError_t e = status_word(&c.status);
  if (e != cudaSuccess) return fail_cuda(e);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  note_other_kernel(s);
  e = launch_norm_rope(c, s);
  return e == cudaSuccess ? TQ_OK : fail_cuda(e);
}

namespace {
int check_sizes(int64_t nseq, int64_t ntok, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                int64_t max_q, int64_t max_kv, int64_t window) {
  if (nseq < 0 || nseq > kMaxPositions || ntok < 0 || ntok > 0x7fffffff || q_heads < 1 ||
      q_heads > 65535 || kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 8 ||
      head_dim % 8 != 0 || head_dim > kMaxKvDim || max_q < 0 || max_q > 0x7fffffff ||
      max_kv < 0 || max_kv > 0x7fffffff || window < 0 ||
      (ntok + 1) * (q_heads / kv_heads) > kMaxPositions - 1024)
    return TQ_ERR_SHAPE;
  return TQ_OK;
}
}  // namespace

int64_t tq_paged_attention_workspace_bytes(int64_t nseq, int64_t ntok, int64_t q_heads,
                                           int64_t kv_heads, int64_t head_dim, int64_t max_q,
                                           int64_t max_kv, int64_t window) {
  if (check_sizes(nseq, ntok, q_heads, kv_heads, head_dim, max_q, max_kv, window) != TQ_OK) return -1;
  if (nseq == 0 || ntok == 0) return 0;
  return attn_plan(nseq, ntok, q_heads, kv_heads, head_dim, max_q, max_kv, window).ws_bytes;
}

int tq_paged_attention(const void* Q, int64_t q_stride, const tq_paged_kv* kv,
                       const int32_t* q_start, const int32_t* kv_len, void* O, int64_t o_stride,
                       int o_type, float* lse, int64_t ntok, int64_t q_heads, int64_t max_q,
                       int64_t max_kv, float scale, int64_t window, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  int rc = check_cache(kv);
  if (rc != TQ_OK) return rc;
  const int64_t dim = kv->head_dim, row = q_heads * dim;
  rc = check_sizes(kv->nseq, ntok, q_heads, kv->heads, dim, max_q, max_kv, window);
  if (rc != TQ_OK) return rc;
  if (!size_ok(q_stride) || !size_ok(o_stride) || !span_ok(ntok, q_stride) ||
      !span_ok(ntok, o_stride) || !std::isfinite(scale))
    return TQ_ERR_SHAPE;
  if (ntok > 1 && (q_stride < row || o_stride < row || q_stride % 8 != 0)) return TQ_ERR_SHAPE;
  if (!type_ok(o_type)) return TQ_ERR_TYPE;
  if (ntok == 0 || kv->nseq == 0) return TQ_OK;
  if (!Q || !O || !q_start || !kv_len) return TQ_ERR_NULL;
  rc = check_cache_pointers(*kv);
  if (rc != TQ_OK) return rc;
  if (!aligned(Q, 16) || !aligned(O, type_bytes(o_type)) || !aligned(q_start, 4) ||
      !aligned(kv_len, 4) || !aligned(lse, 4))
    return TQ_ERR_ALIGN;
  AttnCall c = {};
  c.plan = attn_plan(kv->nseq, ntok, q_heads, kv->heads, dim, max_q, max_kv, window);
  const int64_t need = c.plan.ws_bytes;
  if (need > 0) {
    if (!workspace) return TQ_ERR_NULL;
    if (!aligned(workspace, 16)) return TQ_ERR_ALIGN;
    if (workspace_bytes < need) return TQ_ERR_WORKSPACE;
  }
  const Range in[] = {range(Q, rows_bytes(ntok, q_stride, q_heads, dim, kv->type)),
                      range(kv->k, cache_bytes(*kv)), range(kv->v, cache_bytes(*kv)),
                      range(q_start, (kv->nseq + 1) * 4), range(kv_len, kv->nseq * 4),
                      range(kv->block_table, ((kv->nseq - 1) * kv->table_stride + kv->table_width) * 4)};
  const Range out[] = {range(O, rows_bytes(ntok, o_stride, q_heads, dim, o_type)),
                       range(lse, ntok * q_heads * 4), range(workspace, need)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return TQ_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return TQ_ERR_ALIAS;
  }
  c.q = Q;
  c.q_stride = q_stride;
  c.kv = *kv;
  c.q_start = q_start;
  c.kv_len = kv_len;
  c.o = O;
  c.o_stride = o_stride;
  c.o_type = o_type;
  c.lse = lse;
  c.ntok = ntok;
  c.q_heads = q_heads;
  c.max_q = max_q;
  c.max_kv = max_kv;
  c.scale = scale;
  c.window = window;
  if (need > 0) {
    c.part_o = static_cast<float*>(workspace);
    c.part_lse = c.part_o + c.plan.part_rows * dim;
    if (c.plan.chunk) c.cuts = static_cast<char*>(workspace) + (need - c.plan.blocks * kCutBytes);
  }
  cudaError_t e = status_word(&c.status);
  if (e != cudaSuccess) return fail_cuda(e);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  note_other_kernel(s);
  e = launch_attention(c, s);
  return e == cudaSuccess ? TQ_OK : fail_cuda(e);
}

}  // extern "C"
