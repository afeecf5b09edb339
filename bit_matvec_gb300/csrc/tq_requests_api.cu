// tq_requests_api.cu -- the C ABI of the adapter and sampling calls: argument
// checks, error reporting.
#include "tq_requests.cuh"

namespace tq {
namespace {

bool type_ok(int t) { return t == TQ_F32 || t == TQ_F16 || t == TQ_BF16; }
int64_t type_bytes(int t) { return t == TQ_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0; }

constexpr int64_t kMaxStride = int64_t(1) << 40;
bool stride_ok(int64_t n) { return n >= 0 && n <= kMaxStride; }

// Whether n rows `stride` apart span at most 2^58 values: no memory holds more,
// and sums of such products stay in 64 bits.
bool span_ok(int64_t n, int64_t stride) { return n <= 1 || stride <= (int64_t(1) << 58) / (n - 1); }

int fail_cuda(cudaError_t e) {
  record_cuda_error(e);
  return TQ_ERR_CUDA;
}

struct Range {
  const char* p;
  int64_t n;
};
// n rows of `width` values, `stride` apart.
Range range(const void* p, int64_t n, int64_t stride, int64_t width, int64_t bytes) {
  return {static_cast<const char*>(p), p && n > 0 && width > 0 ? ((n - 1) * stride + width) * bytes : 0};
}
Range range(const void* p, int64_t bytes) { return {static_cast<const char*>(p), p ? bytes : 0}; }
bool overlap(Range a, Range b) {
  return a.n > 0 && b.n > 0 && a.p < b.p + b.n && b.p < a.p + a.n;
}

// Whether rows of two strided buffers overlap: buffers of the same row stride
// whose rows lie side by side in one allocation do not.
bool rows_overlap(Range a, int64_t a_row, Range b, int64_t b_row, int64_t stride, bool same_stride,
                  int64_t n) {
  if (!overlap(a, b)) return false;
  if (!same_stride || n == 1 || stride == 0) return true;
  int64_t d = ((intptr_t)b.p - (intptr_t)a.p) % stride;
  if (d < 0) d += stride;
  return d < a_row || d + b_row > stride;
}

int check_lora(const tq_lora* l) {
  if (!l) return TQ_ERR_NULL;
  if (l->adapters < 0 || l->adapters > kMaxAdapters || l->max_rank < 0 || l->max_rank > kMaxRank ||
      l->rows < 0 || l->rows > kMaxSide || l->cols < 0 || l->cols > kMaxSide || l->cols % 8 != 0)
    return TQ_ERR_SHAPE;
  for (int64_t s : {l->a_stride, l->a_row_stride, l->b_stride, l->b_row_stride})
    if (!stride_ok(s)) return TQ_ERR_SHAPE;
  if (l->a_stride % 8 != 0 || l->a_row_stride % 8 != 0) return TQ_ERR_SHAPE;
  if ((l->max_rank > 1 && l->a_row_stride < l->cols) || (l->rows > 1 && l->b_row_stride < l->max_rank))
    return TQ_ERR_SHAPE;
  if (!span_ok(l->adapters, l->a_stride) || !span_ok(l->adapters, l->b_stride) ||
      !span_ok(l->max_rank, l->a_row_stride) || !span_ok(l->rows, l->b_row_stride))
    return TQ_ERR_SHAPE;
  if (l->type != TQ_F16 && l->type != TQ_BF16) return TQ_ERR_TYPE;
  return TQ_OK;
}

// From the first to the last value of all adapters' A or B.
Range weights(const void* p, const tq_lora& l, int64_t stride, int64_t n, int64_t row_stride, int64_t width) {
  if (l.adapters < 1 || n < 1 || width < 1) return {nullptr, 0};
  return range(p, ((l.adapters - 1) * stride + (n - 1) * row_stride + width) * 2);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

int64_t tq_lora_add_workspace_bytes(int64_t ntok, int64_t adapters) {
  if (ntok < 0 || ntok > 0x7fffffff || adapters < 0 || adapters > kMaxAdapters) return -1;
  return lora_workspace_bytes(ntok, adapters);
}

int tq_lora_add(const void* X, int64_t x_stride, int x_type, const tq_lora* lora, const int32_t* ids,
                const void* Z, int64_t z_stride, void* Y, int64_t y_stride, int y_type, int64_t ntok,
                void* workspace, int64_t workspace_bytes, void* stream) {
  int rc = check_lora(lora);
  if (rc != TQ_OK) return rc;
  const tq_lora& l = *lora;
  if (ntok < 0 || ntok > 0x7fffffff) return TQ_ERR_SHAPE;
  for (int64_t s : {x_stride, z_stride, y_stride})
    if (!stride_ok(s) || !span_ok(ntok, s)) return TQ_ERR_SHAPE;
  if (!type_ok(y_type) || (x_type != TQ_F32 && x_type != l.type)) return TQ_ERR_TYPE;
  const int64_t xb = type_bytes(x_type), yb = type_bytes(y_type);
  if (ntok > 1 && (x_stride < l.cols || x_stride * xb % 16 != 0 || y_stride < l.rows ||
                   (Z && z_stride < l.rows)))
    return TQ_ERR_SHAPE;
  if (ntok == 0 || l.rows == 0) return TQ_OK;
  // (without columns h is zeros, and B is multiplied by them all the same)
  const bool work = l.adapters > 0 && l.max_rank > 0;
  if (!ids || !Y || (work && (!l.b || (l.cols > 0 && (!X || !l.a))))) return TQ_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(Y, yb) || !aligned(Z, yb) || !aligned(X, 16) || !aligned(l.a, 16) ||
      !aligned(l.b, 2) || !aligned(l.rank, 4) || !aligned(l.scale, 4))
    return TQ_ERR_ALIGN;
  const int64_t need = lora_workspace_bytes(ntok, l.adapters);
  if (need > 0) {
    if (!workspace) return TQ_ERR_NULL;
    if (!aligned(workspace, 16)) return TQ_ERR_ALIGN;
    if (workspace_bytes < need) return TQ_ERR_WORKSPACE;
  }
  const Range x = range(X, ntok, x_stride, l.cols, xb), z = range(Z, ntok, z_stride, l.rows, yb);
  const Range y = range(Y, ntok, y_stride, l.rows, yb), w = range(workspace, need);
  const Range in[] = {weights(l.a, l, l.a_stride, l.max_rank, l.a_row_stride, l.cols),
                      weights(l.b, l, l.b_stride, l.rows, l.b_row_stride, l.max_rank),
                      range(l.rank, l.adapters * 4), range(l.scale, l.adapters * 4), range(ids, ntok * 4)};
  for (const Range& r : in)
    if (overlap(y, r) || overlap(w, r)) return TQ_ERR_ALIAS;
  if (overlap(w, x) || overlap(w, y) || overlap(w, z)) return TQ_ERR_ALIAS;
  if (rows_overlap(y, l.rows * yb, x, l.cols * xb, y_stride * yb, y_stride * yb == x_stride * xb, ntok))
    return TQ_ERR_ALIAS;
  const bool in_place = Z == Y && (z_stride == y_stride || ntok == 1);
  if (!in_place && rows_overlap(y, l.rows * yb, z, l.rows * yb, y_stride * yb, y_stride == z_stride, ntok))
    return TQ_ERR_ALIAS;
  LoraCall c = {X, x_stride, x_type, l, ids, Z, z_stride, Y, y_stride, y_type, ntok, workspace, nullptr};
  cudaError_t e = status_word(&c.status);
  if (e != cudaSuccess) return fail_cuda(e);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  note_other_kernel(s);
  e = launch_lora_add(c, s);
  return e == cudaSuccess ? TQ_OK : fail_cuda(e);
}

int tq_sample(const void* logits, int64_t stride, int type, int64_t ntok, int64_t vocab, const float* u,
              const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
              int32_t* tokens, float* logp, void* stream) {
  if (ntok < 0 || ntok > 0x7fffffff || vocab < 1 || vocab > kMaxVocab || !stride_ok(stride) ||
      !span_ok(ntok, stride) || (ntok > 1 && stride < vocab))
    return TQ_ERR_SHAPE;
  if (!type_ok(type)) return TQ_ERR_TYPE;
  if (ntok == 0) return TQ_OK;
  if (!logits || !u || !tokens) return TQ_ERR_NULL;
  if (!aligned(logits, type_bytes(type))) return TQ_ERR_ALIGN;
  for (const void* p : {(const void*)u, (const void*)temperature, (const void*)top_k, (const void*)top_p,
                        (const void*)min_p, (const void*)tokens, (const void*)logp})
    if (!aligned(p, 4)) return TQ_ERR_ALIGN;
  const Range in[] = {range(logits, ntok, stride, vocab, type_bytes(type)), range(u, ntok * 4),
                      range(temperature, ntok * 4), range(top_k, ntok * 4), range(top_p, ntok * 4),
                      range(min_p, ntok * 4)};
  const Range out[] = {range(tokens, ntok * 4), range(logp, ntok * 4)};
  for (const Range& r : in)
    if (overlap(out[0], r) || overlap(out[1], r)) return TQ_ERR_ALIAS;
  if (overlap(out[0], out[1])) return TQ_ERR_ALIAS;
  const SampleCall c = {logits, stride, type, ntok, (int)vocab, u, temperature, top_k, top_p, min_p,
                        tokens, logp};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  note_other_kernel(s);
  const cudaError_t e = launch_sample(c, s);
  return e == cudaSuccess ? TQ_OK : fail_cuda(e);
}

}  // extern "C"
