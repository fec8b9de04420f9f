// q8_heads_f32.cu -- the heads' kernels of fp32 values.
#include "q8_heads.cuh"

namespace c3d {

template cudaError_t launch_heads_in<float>(const HeadsParams&, int, bool, cudaStream_t);

}  // namespace c3d
