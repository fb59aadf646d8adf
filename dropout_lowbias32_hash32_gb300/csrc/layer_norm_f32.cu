// layer_norm_f32.cu -- the layer-norm kernels for f32 rows.
#include "layer_norm_kernels.cuh"

namespace rngk {
template cudaError_t launch_norm_fwd<float, float>(const NormFwd &, bool, cudaStream_t);
template cudaError_t launch_norm_bwd<float, float>(const NormBwd &, bool, cudaStream_t);
template cudaError_t stalled_waits_norm<float>(uint64_t *);
}  // namespace rngk
