// tensor_map.h -- TMA descriptors of [batch, length, heads, head_dim] arrays.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attention.h"

namespace rngk {

// cuTensorMapEncodeTiled, from the driver that the runtime has loaded; null
// when it has none.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A box of box_len positions of one head (or, with pack heads side by side,
// box_len / pack positions of each) by 64 elements, read as box_len rows of 128
// bytes with the 128-byte swizzle.  Dimensions: element, head in its pack,
// position, pack, batch.  What lies outside the array reads as zero.
inline cudaError_t make_heads_map(CUtensorMap *map, bool bf16, const void *p, const Strides &s, int32_t batch,
                                  int32_t len, int32_t heads, int32_t dim, int32_t pack, int32_t box_len)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t sizes[5] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(pack),
                                 static_cast<cuuint64_t>(len), static_cast<cuuint64_t>(heads / pack),
                                 static_cast<cuuint64_t>(batch)};
    // a stride along a size of 1 is never used, but is looked at
    auto bytes = [](int64_t stride, int64_t n) { return static_cast<cuuint64_t>(n > 1 ? 2 * stride : 16); };
    const cuuint64_t strides[4] = {bytes(s.head, pack), bytes(s.len, len), bytes(s.head * pack, heads / pack),
                                   bytes(s.batch, batch)};
    const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(pack), static_cast<cuuint32_t>(box_len / pack), 1, 1};
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    const CUresult r = encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                              const_cast<void *>(p), sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace rngk
