// pa_rope_axes.cu -- the rotary append by positions of the rows' own on one or more axes (kernels:
// pa_rope.cuh).  The rows of a drafted tree turn by their depth while they lie one behind the other,
// those of an image by its time, height and width.
#include "pa_rope.cuh"

namespace pa {

cudaError_t launch_rope_append_axes(const RopeArgs& a, cudaStream_t stream) { return launch_rows<true>(a, stream); }

}  // namespace pa
