// layer_norm_f16.cu -- the layer-norm kernels for f16 rows.
#include "layer_norm_kernels.cuh"

namespace rngk {
template cudaError_t launch_norm_fwd<__half, __half>(const NormFwd &, bool, cudaStream_t);
template cudaError_t launch_norm_bwd<__half, __half>(const NormBwd &, bool, cudaStream_t);
template cudaError_t launch_norm_fwd<__half, float>(const NormFwd &, bool, cudaStream_t);
template cudaError_t launch_norm_bwd<__half, float>(const NormBwd &, bool, cudaStream_t);
template cudaError_t stalled_waits_norm<__half>(uint64_t *);
}  // namespace rngk
