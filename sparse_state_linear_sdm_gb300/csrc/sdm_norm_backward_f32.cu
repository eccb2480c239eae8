// Gradient of the norms: the instances of fp32.
#include "sdm_norm_backward.cuh"

namespace sdm {
template int launch_norm_backward<float, float>(const NormBackward&, int, bool, cudaStream_t);
}  // namespace sdm
