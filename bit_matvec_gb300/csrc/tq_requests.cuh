// tq_requests.cuh -- internals of the operators that differ from request to
// request: low-rank adapters beside a product, and the draw of the next token.
// Nothing here is visible outside the library.
#pragma once

#include "tq_attn.cuh"

namespace tq {

constexpr int64_t kMaxAdapters = 32768;
constexpr int64_t kMaxRank = 256;
constexpr int64_t kMaxSide = int64_t(1) << 24;    // rows and columns of an adapted matrix
constexpr int kMaxVocab = 1 << 18;

struct LoraCall {
  const void* x;
  int64_t x_stride;
  int x_type;
  tq_lora lora;
  const int32_t* ids;
  const void* z;
  int64_t z_stride;
  void* y;
  int64_t y_stride;
  int y_type;
  int64_t ntok;
  void* ws;
  int* status;
};
cudaError_t launch_lora_add(const LoraCall& c, cudaStream_t s);
int64_t lora_workspace_bytes(int64_t ntok, int64_t adapters);

struct SampleCall {
  const void* logits;
  int64_t stride;
  int type;
  int64_t ntok;
  int vocab;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logp;
};
cudaError_t launch_sample(const SampleCall& c, cudaStream_t s);

}  // namespace tq
