// layer_norm.h -- what the layer-norm kernels are launched with (host side of
// layer_norm.cu, kernels in layer_norm_kernels.cuh).
#pragma once

#include "element.cuh"
#include "internal.h"

namespace rngk {

template <class T>
struct Rows {
    T *p;
    size_t stride;
};

struct NormFwd {
    Rows<const void> x, residual;
    Rows<void> y, h;
    const void *bias, *gamma, *beta;
    float *mean, *rstd;
    size_t rows;
    uint32_t cols;
    float eps;
    uint32_t first;
    Mask mask;
};

struct NormBwd {
    Rows<const void> dy, h, dh;
    Rows<void> dx, dresidual;
    const void *gamma;
    const float *mean, *rstd;
    void *dgamma, *dbeta, *dbias;
    size_t rows;
    uint32_t cols;
    uint32_t first;
    Mask mask;
    float *workspace;
};

// Elements of one vector access of the rows: 16 bytes, or 1 when a row or an
// address is not on that boundary.
template <class T, class W>
cudaError_t launch_norm_fwd(const NormFwd &a, bool vectors, cudaStream_t s);
template <class T, class W>
cudaError_t launch_norm_bwd(const NormBwd &a, bool vectors, cudaStream_t s);

// Waits that ran out in the kernels for T, on the current device.
template <class T>
cudaError_t stalled_waits_norm(uint64_t *count);

// How the backward pass is cut: the fused kernel's blocks (group threads share
// a row of cols columns, per_block rows at a time), its form with a ring's
// (ring_group threads to a row, ring_per_sm blocks to an SM), or for long rows
// the two-kernel form's chunks of rows.
struct NormBwdPlan {
    bool fused;
    unsigned group, per_block, blocks, ring_group, ring_per_sm, ring_blocks;
    size_t workspace_floats;
};
NormBwdPlan norm_bwd_plan(size_t rows, size_t cols);

}  // namespace rngk
