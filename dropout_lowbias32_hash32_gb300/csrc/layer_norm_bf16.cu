// layer_norm_bf16.cu -- the layer-norm kernels for bf16 rows.
#include "layer_norm_kernels.cuh"

namespace rngk {
template cudaError_t launch_norm_fwd<__nv_bfloat16, __nv_bfloat16>(const NormFwd &, bool, cudaStream_t);
template cudaError_t launch_norm_bwd<__nv_bfloat16, __nv_bfloat16>(const NormBwd &, bool, cudaStream_t);
template cudaError_t launch_norm_fwd<__nv_bfloat16, float>(const NormFwd &, bool, cudaStream_t);
template cudaError_t launch_norm_bwd<__nv_bfloat16, float>(const NormBwd &, bool, cudaStream_t);
template cudaError_t stalled_waits_norm<__nv_bfloat16>(uint64_t *);
}  // namespace rngk
