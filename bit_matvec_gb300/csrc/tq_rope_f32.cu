// tq_rope_f32.cu -- norm and rotation of f32 heads (see tq_rope.cuh).
#include "tq_rope.cuh"

namespace tq {

cudaError_t launch_norm_rope_f32(const RopeCall& c, cudaStream_t s) { return launch_out<float>(c, s); }

}  // namespace tq
