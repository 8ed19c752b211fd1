// pa_rope.cu -- the rotary append by the rows' place in their sequence (kernels: pa_rope.cuh).
#include "pa_rope.cuh"

namespace pa {

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream) { return launch_rows<false>(a, stream); }

}  // namespace pa
