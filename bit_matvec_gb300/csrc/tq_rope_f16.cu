// tq_rope_f16.cu -- norm and rotation of f16 heads (see tq_rope.cuh).
#include "tq_rope.cuh"

namespace tq {

cudaError_t launch_norm_rope_f16(const RopeCall& c, cudaStream_t s) { return launch_out<__half>(c, s); }

}  // namespace tq
