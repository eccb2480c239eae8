// Gradient of the norms: the instances of bf16 with an fp32 residual stream.
#include "sdm_norm_backward.cuh"

namespace sdm {
template int launch_norm_backward<__nv_bfloat16, float>(const NormBackward&, int, bool, cudaStream_t);
}  // namespace sdm
