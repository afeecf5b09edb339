// tq_rope_bf16.cu -- norm and rotation of bf16 heads (see tq_rope.cuh).
#include "tq_rope.cuh"

namespace tq {

cudaError_t launch_norm_rope_bf16(const RopeCall& c, cudaStream_t s) { return launch_out<__nv_bfloat16>(c, s); }

}  // namespace tq
