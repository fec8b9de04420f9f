// q8_heads_f16.cu -- the heads' kernels of fp16 values.
#include "q8_heads.cuh"

namespace c3d {

template cudaError_t launch_heads_in<__half>(const HeadsParams&, int, bool, cudaStream_t);

}  // namespace c3d
