// layer_norm_kernels.cuh -- bias + dropout + residual + layer norm, forward
// and backward (include/rng.h, rng_dropout_layer_norm_*).  Included by one
// translation unit per element type.
//
// Bound by HBM: the forward pass reads x and residual and writes y and h (8
// bytes an element in 16-bit types), the backward pass reads dy, h, dh and
// writes dx, dresidual (10 bytes), for 40 instructions an element, about ten of
// them the mask's hash.  So a row is read once and stays in registers (or shared
// memory) between its reductions; the mask is redrawn from the element's flat
// index.  Measured, 16384 x 4096 in bf16, p = 0.1: forward 92 us, 537 MB at 5.9
// TB/s, issue slots 77 % busy; backward 123 us, 671 MB at 5.4 TB/s, of which the
// sums of the weights' gradients 7 us.  2^20 x 256 in f32, forward: 615 us, 4.3 GB
// at 7.0 TB/s.  Rows off a vector boundary and, backward, of more than 8192
// columns take an element an access: 1531 x 769 in f16, backward, 24 us for 11.8 MB.
#pragma once

#include "barrier.cuh"
#include "layer_norm.h"

namespace rngk {
namespace {

// Sums over a row's threads: a warp, or the whole block with one barrier a
// call (consecutive calls alternate between two halves of `scratch`, so the
// reads of one need no barrier before the writes of the next).
template <bool kWarp, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float *scratch, uint32_t &phase)
{
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], m);
    if constexpr (!kWarp) {
        const uint32_t warps = blockDim.x / 32u, warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
        float *half = scratch + phase * (32u * K);
        phase ^= 1u;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) half[32u * k + warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = lane < warps ? half[32u * k + lane] : 0.0f;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], m);
    }
}

template <class T>
__device__ __forceinline__ const T *row_of(const Rows<const void> &a, size_t row)
{
    return static_cast<const T *>(a.p) + row * a.stride;
}
template <class T>
__device__ __forceinline__ T *row_of(const Rows<void> &a, size_t row)
{
    return static_cast<T *>(a.p) + row * a.stride;
}

// h of V adjacent elements: residual + dropout(x + bias).
template <class T, class W, int V>
__device__ __forceinline__ void hidden(const NormFwd &a, const Raw<T, V> &x, const Raw<T, V> &res, uint32_t col,
                                       uint32_t c, float (&h)[V])
{
    unpack<T, V>(x, h);
    if (a.bias) {
        float b[V];
        unpack<W, V>(load<false, W, V>(static_cast<const W *>(a.bias) + col), b);
        add_all<V>(h, h, b);
    }
    if (a.mask.threshold) drop_all<V>(a.mask, c, h);
    if (a.residual.p) {
        float r[V];
        unpack<T, V>(res, r);
        add_all<V>(h, h, r);
    }
}

// y of V adjacent elements.
template <class W, int V>
__device__ __forceinline__ void normalised(const NormFwd &a, const float (&h)[V], float mean, float rstd, uint32_t col,
                                           float (&y)[V])
{
    // h rstd - mean rstd would cancel where the mean is far above the deviations: the difference first
    fma_all<V>(y, h, 1.0f, -mean);
    float g[V];
    unpack<W, V>(load_or_one<W, V>(a.gamma, col), g);
    fma_all<V>(g, g, rstd, 0.0f);
    if (a.beta) {
        float b[V];
        unpack<W, V>(load<false, W, V>(static_cast<const W *>(a.beta) + col), b);
        fma_all<V>(y, y, g, b);
    } else {
        mul_all<V>(y, y, g);
    }
}

// Mean and sum of squared deviations of a row of n elements, of which the
// thread has e[0 .. count).  A warp takes both over its own elements, the
// deviations from its own mean, in two rounds of shuffles; the block's warps
// are then joined with one barrier: with m the mean of the whole, a part of n_w
// elements contributes n_w (m_w - m)^2 to the deviations beside its own sum.
struct Moments {
    float mean, deviations;
};
template <bool kWarp, int V, int P>
__device__ __forceinline__ Moments row_moments(const float (&h)[P][V], uint32_t vectors, float2 *scratch)
{
    const uint32_t group = blockDim.x, t = threadIdx.x;
    auto share = [&](uint32_t warp) {  // elements of a warp of the row's
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t first = 32u * warp + i * group;
            n += first < vectors ? min(vectors - first, 32u) : 0u;
        }
        return static_cast<float>(n * V);
    };
    auto warp_sum = [](float v) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
        return v;
    };
    const uint32_t warp = kWarp ? 0u : t / 32u;
    const float mine = share(warp);
    float sum[V] = {}, squares[V] = {};
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (t + i * group < vectors) add_all<V>(sum, sum, h[i]);
#pragma unroll
    for (int k = 1; k < V; ++k) sum[0] += sum[k];
    Moments m;
    m.mean = mine > 0.0f ? warp_sum(sum[0]) / mine : 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (t + i * group < vectors) {
            float d[V];
            fma_all<V>(d, h[i], 1.0f, -m.mean);
            fma_all<V>(squares, d, d, squares);
        }
#pragma unroll
    for (int k = 1; k < V; ++k) squares[0] += squares[k];
    m.deviations = warp_sum(squares[0]);
    if constexpr (!kWarp) {
        const uint32_t lane = t % 32u;
        if (lane == 0) scratch[warp] = make_float2(m.mean, m.deviations);
        __syncthreads();
        const float n = lane < group / 32u ? share(lane) : 0.0f;
        const float2 part = n > 0.0f ? scratch[lane] : make_float2(0.0f, 0.0f);
        m.mean = warp_sum(n * part.x) / static_cast<float>(vectors * V);
        m.deviations = warp_sum(part.y + n * (part.x - m.mean) * (part.x - m.mean));
    }
    return m;
}

// Rows held in registers: blockDim.x threads share a row (kWarp: a warp, and
// blockDim.y rows to a block), each with P vectors of V elements.
template <class T, class W, int V, int P, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : 1024) norm_fwd_kernel(const __grid_constant__ NormFwd a)
{
    __shared__ float2 scratch[32];
    const size_t row = static_cast<size_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (kWarp && row >= a.rows) return;
    const uint32_t group = blockDim.x, vectors = a.cols / V, t = threadIdx.x;
    const uint32_t c0 = a.first + static_cast<uint32_t>(row) * a.cols;

    Raw<T, V> x[P], res[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const uint32_t v = t + i * group;
        if (v < vectors) x[i] = load<true, T, V>(row_of<T>(a.x, row) + v * V);
    }
    if (a.residual.p) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t v = t + i * group;
            if (v < vectors) res[i] = load<true, T, V>(row_of<T>(a.residual, row) + v * V);
        }
    }
    float h[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const uint32_t v = t + i * group;
        if (v < vectors) hidden<T, W, V>(a, x[i], res[i], v * V, c0 + v * V, h[i]);
    }
    const Moments m = row_moments<kWarp, V, P>(h, vectors, scratch);
    const float mean = m.mean, rstd = 1.0f / sqrtf(m.deviations / static_cast<float>(a.cols) + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const uint32_t v = t + i * group;
        if (v < vectors) {
            if (a.h.p) store<T, V>(row_of<T>(a.h, row) + v * V, h[i]);
            float y[V];
            normalised<W, V>(a, h[i], mean, rstd, v * V, y);
            store<T, V>(row_of<T>(a.y, row) + v * V, y);
        }
    }
}

// Rows too long for registers: three passes over the row, the second and third
// out of L2, one element at a time.  An element's h and y are written by the
// thread that last read its x and residual, so in place is fine.
template <class T, class W>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const __grid_constant__ NormFwd a)
{
    __shared__ float scratch[64];
    uint32_t phase = 0;
    const size_t row = blockIdx.x;
    const uint32_t c0 = a.first + static_cast<uint32_t>(row) * a.cols;
    auto hidden_at = [&](uint32_t j) {
        const Raw<T, 1> x = load<false, T, 1>(row_of<T>(a.x, row) + j);
        Raw<T, 1> res{};
        if (a.residual.p) res = load<false, T, 1>(row_of<T>(a.residual, row) + j);
        float h[1];
        hidden<T, W, 1>(a, x, res, j, c0 + j, h);
        return h[0];
    };
    float sum[1] = {0.0f}, square[1] = {0.0f};
    for (uint32_t j = threadIdx.x; j < a.cols; j += blockDim.x) sum[0] += hidden_at(j);
    row_sum<false, 1>(sum, scratch, phase);
    const float mean = sum[0] / static_cast<float>(a.cols);
    for (uint32_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
        const float d = hidden_at(j) - mean;
        square[0] += d * d;
    }
    row_sum<false, 1>(square, scratch, phase);
    const float rstd = 1.0f / sqrtf(square[0] / static_cast<float>(a.cols) + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    for (uint32_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
        const float h[1] = {hidden_at(j)};
        if (a.h.p) store<T, 1>(row_of<T>(a.h, row) + j, h);
        float y[1];
        normalised<W, 1>(a, h, mean, rstd, j, y);
        store<T, 1>(row_of<T>(a.y, row) + j, y);
    }
}

// ---- backward ---------------------------------------------------------------

constexpr int kBwdElems = 8;  // elements of a row in one thread's registers

// One kernel for rows of up to 8192 columns: blockDim.x threads hold a row,
// eight elements each, and a block walks the rows blockIdx.x, + gridDim.x, ...
// (times blockDim.y when a warp holds a row).  The three column sums stay in
// the threads' registers over the walk, so dy, h and dh are read once; a block
// writes one row of partial sums, which column_sum_kernel adds up in a fixed
// order.
constexpr uint32_t kRingStages = 8;
constexpr int kRingElems = 16;

template <class T, class W, int V, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 256 : 1024) norm_bwd_kernel(const __grid_constant__ NormBwd a)
{
    constexpr int P = kBwdElems / V;
    __shared__ float scratch[kWarp ? 8 * 32 * kBwdElems : 128];
    uint32_t phase = 0;
    const uint32_t group = blockDim.x, vectors = a.cols / V, t = threadIdx.x;
    const float inv = 1.0f / static_cast<float>(a.cols);
    float dgamma[P][V] = {}, dbeta[P][V] = {}, dbias[P][V] = {};

    for (size_t row = static_cast<size_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows;
         row += static_cast<size_t>(gridDim.x) * blockDim.y) {
        const uint32_t c0 = a.first + static_cast<uint32_t>(row) * a.cols;
        const float mean = a.mean[row], rstd = a.rstd[row];
        Raw<T, V> dy_raw[P], h_raw[P], dh_raw[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t v = t + i * group;
            if (v < vectors) {
                dy_raw[i] = load<true, T, V>(row_of<T>(a.dy, row) + v * V);
                h_raw[i] = load<true, T, V>(row_of<T>(a.h, row) + v * V);
                if (a.dh.p) dh_raw[i] = load<true, T, V>(row_of<T>(a.dh, row) + v * V);
            }
        }
        float g[P][V], n[P][V], sums[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t v = t + i * group;
            if (v < vectors) {
                unpack<T, V>(dy_raw[i], g[i]);
                unpack<T, V>(h_raw[i], n[i]);
                float w[V];
                if (a.gamma) unpack<W, V>(load<false, W, V>(static_cast<const W *>(a.gamma) + v * V), w);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    n[i][k] = (n[i][k] - mean) * rstd;
                    dgamma[i][k] += g[i][k] * n[i][k];
                    dbeta[i][k] += g[i][k];
                    if (a.gamma) g[i][k] *= w[k];
                    sums[0] += g[i][k];
                    sums[1] += g[i][k] * n[i][k];
                }
            }
        }
        row_sum<kWarp, 2>(sums, scratch, phase);
        const float m0 = sums[0] * inv, m1 = sums[1] * inv;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t v = t + i * group;
            if (v < vectors) {
                float dz[V];
#pragma unroll
                for (int k = 0; k < V; ++k) dz[k] = rstd * (g[i][k] - m0 - n[i][k] * m1);
                if (a.dh.p) {
                    float d[V];
                    unpack<T, V>(dh_raw[i], d);
#pragma unroll
                    for (int k = 0; k < V; ++k) dz[k] += d[k];
                }
                if (a.dresidual.p) store<T, V>(row_of<T>(a.dresidual, row) + v * V, dz);
                if (a.mask.threshold) drop_all<V>(a.mask, c0 + v * V, dz);
#pragma unroll
                for (int k = 0; k < V; ++k) dbias[i][k] += dz[k];
                store<T, V>(row_of<T>(a.dx, row) + v * V, dz);
            }
        }
    }

    float *part = a.workspace + static_cast<size_t>(blockIdx.x) * 3u * a.cols;
    auto put = [&](float (&s)[P][V], float *out) {
        if constexpr (kWarp) {  // the block's warps, in order
            __syncthreads();
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) scratch[(threadIdx.y * kBwdElems + i * V + k) * 32 + t] = s[i][k];
            __syncthreads();
            if (threadIdx.y) return;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    for (uint32_t w = 1; w < blockDim.y; ++w) s[i][k] += scratch[(w * kBwdElems + i * V + k) * 32 + t];
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t v = t + i * group;
            if (v < vectors) {
#pragma unroll
                for (int k = 0; k < V; ++k) out[v * V + k] = s[i][k];
            }
        }
    };
    put(dgamma, part);
    put(dbeta, part + a.cols);
    put(dbias, part + 2u * a.cols);
}

// The same for rows of whole 16-byte vectors that a block shares: rows to come
// are copied to a ring in shared memory by bulk copies, so that the loads of
// some rows are under way behind the reduction of one (a row's own loads,
// then its barrier, then its stores left HBM idle).  Sixteen elements to a thread:
// a thread's share of the reduction and the addresses costs as much as ten.
template <class T, class W, int V>
__global__ void __launch_bounds__(512) norm_bwd_ring_kernel(const __grid_constant__ NormBwd a, uint32_t stages)
{
    constexpr int P = kRingElems / V;
    extern __shared__ uint4 ring[];  // [stages][dy, h, dh]
    __shared__ alignas(8) uint64_t bars[kRingStages];
    __shared__ float scratch[128];
    __shared__ volatile uint32_t stalled;
    uint32_t phase = 0;
    const uint32_t group = blockDim.x, vectors = a.cols / V, t = threadIdx.x, full = smem_address(bars);
    const uint32_t row_bytes = a.cols * sizeof(T), arrays = a.dh.p ? 3u : 2u, stage_bytes = arrays * row_bytes;
    const float inv = 1.0f / static_cast<float>(a.cols);
    auto fetch = [&](uint32_t n, uint32_t stage) {  // the block's n-th row, by one thread
        const size_t row = blockIdx.x + static_cast<size_t>(n) * gridDim.x;
        if (row >= a.rows || stalled) return;
        const uint32_t bar = full + 8 * stage, dst = smem_address(ring) + stage * stage_bytes;
        barrier_expect(bar, stage_bytes);
        bulk_load(dst, row_of<T>(a.dy, row), row_bytes, bar);
        bulk_load(dst + row_bytes, row_of<T>(a.h, row), row_bytes, bar);
        if (a.dh.p) bulk_load(dst + 2 * row_bytes, row_of<T>(a.dh, row), row_bytes, bar);
    };
    if (t == 0) {
        stalled = 0;
        for (uint32_t s = 0; s < stages; ++s) barrier_init(full + 8 * s, 1);
        fence_barrier_init();
        for (uint32_t s = 0; s < stages; ++s) fetch(s, s);
    }
    Raw<W, V> gamma[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (t + i * group < vectors) gamma[i] = load_or_one<W, V>(a.gamma, (t + i * group) * V);
    float dgamma[P][V] = {}, dbeta[P][V] = {}, dbias[P][V] = {};
    __syncthreads();

    size_t row = blockIdx.x;
    float mean = a.mean[row], rstd = a.rstd[row];
    uint32_t stage = 0, parity = 0;
    for (uint32_t n = 0; row < a.rows; ++n) {
        const size_t next_row = row + gridDim.x;
        const size_t peek = next_row < a.rows ? next_row : row;
        const float next_mean = a.mean[peek], next_rstd = a.rstd[peek];
        barrier_wait_one(full + 8 * stage, parity, &stalled);
        const T *in = reinterpret_cast<const T *>(reinterpret_cast<const uint8_t *>(ring) + stage * stage_bytes);
        // dy, dy gamma and (h - mean) rstd of a vector
        auto inputs = [&](int i, uint32_t v, float (&dy)[V], float (&g)[V], float (&x)[V]) {
            unpack<T, V>(load<false, T, V>(in + v * V), dy);
            unpack<T, V>(load<false, T, V>(in + a.cols + v * V), x);
            unpack<W, V>(gamma[i], g);
            fma_all<V>(x, x, 1.0f, -mean);
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] *= rstd;
            mul_all<V>(g, g, dy);
        };
        float part0[V] = {}, part1[V] = {};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t v = t + i * group;
            if (v < vectors) {
                float dy[V], g[V], x[V];
                inputs(i, v, dy, g, x);
                fma_all<V>(dgamma[i], dy, x, dgamma[i]);
                add_all<V>(dbeta[i], dbeta[i], dy);
                add_all<V>(part0, part0, g);
                fma_all<V>(part1, g, x, part1);
            }
        }
        float sums[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < V; ++k) sums[0] += part0[k], sums[1] += part1[k];
        row_sum<false, 2>(sums, scratch, phase);
        // every thread has left the previous row behind
        if (t == 0 && n > 0) fence_async_shared(), fetch(n - 1 + stages, stage ? stage - 1 : stages - 1);
        const float m0 = sums[0] * inv, m1 = sums[1] * inv;
        const uint32_t c0 = a.first + static_cast<uint32_t>(row) * a.cols;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t v = t + i * group;
            if (v < vectors) {
                float dy[V], g[V], x[V], dz[V];
                inputs(i, v, dy, g, x);
                fma_all<V>(g, x, -m1, g);
                fma_all<V>(dz, g, 1.0f, -m0);
                if (a.dh.p) {
                    float d[V];
                    unpack<T, V>(load<false, T, V>(in + 2 * a.cols + v * V), d);
                    fma_all<V>(dz, dz, rstd, d);
                } else {
                    fma_all<V>(dz, dz, rstd, 0.0f);
                }
                if (a.dresidual.p) store<T, V>(row_of<T>(a.dresidual, row) + v * V, dz);
                if (a.mask.threshold) drop_all<V>(a.mask, c0 + v * V, dz);
                add_all<V>(dbias[i], dbias[i], dz);
                store<T, V>(row_of<T>(a.dx, row) + v * V, dz);
            }
        }
        row = next_row, mean = next_mean, rstd = next_rstd;
        if (++stage == stages) stage = 0, parity ^= 1u;
    }
    if (stalled && t == 0)  // nothing may land after the block has ended
        for (uint32_t s = 0; s < stages; ++s) barrier_drain(full + 8 * s, 0), barrier_drain(full + 8 * s, 1);

    float *part = a.workspace + static_cast<size_t>(blockIdx.x) * 3u * a.cols;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const uint32_t v = t + i * group;
        if (v < vectors) {
#pragma unroll
            for (int k = 0; k < V; k += 4) {
                float *out = part + v * V + k;
                *reinterpret_cast<float4 *>(out) = make_float4(dgamma[i][k], dgamma[i][k + 1], dgamma[i][k + 2], dgamma[i][k + 3]);
                *reinterpret_cast<float4 *>(out + a.cols) = make_float4(dbeta[i][k], dbeta[i][k + 1], dbeta[i][k + 2], dbeta[i][k + 3]);
                *reinterpret_cast<float4 *>(out + 2 * a.cols) = make_float4(dbias[i][k], dbias[i][k + 1], dbias[i][k + 2], dbias[i][k + 3]);
            }
        }
    }
}

// Rows too long for the fused kernel, first half: the two means of every row.
template <class T, class W>
__global__ void __launch_bounds__(1024) norm_bwd_means_kernel(const __grid_constant__ NormBwd a)
{
    __shared__ float scratch[128];
    uint32_t phase = 0;
    const size_t row = blockIdx.x;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float sums[2] = {0.0f, 0.0f};
    for (uint32_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
        float g = to_f32(row_of<T>(a.dy, row)[j]);
        if (a.gamma) g *= to_f32(static_cast<const W *>(a.gamma)[j]);
        sums[0] += g;
        sums[1] += g * ((to_f32(row_of<T>(a.h, row)[j]) - mean) * rstd);
    }
    row_sum<false, 2>(sums, scratch, phase);
    if (threadIdx.x == 0) {
        a.workspace[2 * row] = sums[0] / static_cast<float>(a.cols);
        a.workspace[2 * row + 1] = sums[1] / static_cast<float>(a.cols);
    }
}

// Second half: one thread a column, block (x, y) over the y-th chunk of rows.
template <class T, class W>
__global__ void __launch_bounds__(256) norm_bwd_columns_kernel(const __grid_constant__ NormBwd a)
{
    const uint32_t j = blockIdx.x * 256u + threadIdx.x;
    if (j >= a.cols) return;
    const size_t chunk = (a.rows + gridDim.y - 1) / gridDim.y;
    const size_t begin = chunk * blockIdx.y, end = begin + chunk < a.rows ? begin + chunk : a.rows;
    const float w = a.gamma ? to_f32(static_cast<const W *>(a.gamma)[j]) : 1.0f;
    float dgamma = 0.0f, dbeta = 0.0f, dbias = 0.0f;
    for (size_t row = begin; row < end; ++row) {
        const float rstd = a.rstd[row], dy = to_f32(row_of<T>(a.dy, row)[j]);
        const float n = (to_f32(row_of<T>(a.h, row)[j]) - a.mean[row]) * rstd;
        float dz = rstd * (dy * w - a.workspace[2 * row] - n * a.workspace[2 * row + 1]);
        if (a.dh.p) dz += to_f32(row_of<T>(a.dh, row)[j]);
        if (a.dresidual.p) row_of<T>(a.dresidual, row)[j] = from_f32<T>(dz);
        if (a.mask.threshold)
            dz = keeps(a.mask, a.first + static_cast<uint32_t>(row) * a.cols + j) ? dz * a.mask.scale : 0.0f;
        row_of<T>(a.dx, row)[j] = from_f32<T>(dz);
        dgamma += dy * n, dbeta += dy, dbias += dz;
    }
    float *part = a.workspace + 2 * a.rows + static_cast<size_t>(blockIdx.y) * 3u * a.cols;
    part[j] = dgamma, part[static_cast<size_t>(a.cols) + j] = dbeta, part[size_t(2) * a.cols + j] = dbias;
}

// The weights' gradients from `blocks` rows of [3][cols] partial sums: a warp
// of adjacent columns adds every 16th row from its own on, then the block's 16
// warps are added in a fixed order.
constexpr uint32_t kSumWarps = 16;
template <class W>
__global__ void __launch_bounds__(32 * kSumWarps) column_sum_kernel(const float *part, uint32_t blocks, uint32_t cols, W *dgamma,
                                                                    W *dbeta, W *dbias)
{
    __shared__ float sums[kSumWarps][32];
    W *out = blockIdx.y == 0 ? dgamma : blockIdx.y == 1 ? dbeta : dbias;
    if (out == nullptr) return;
    const uint32_t j = blockIdx.x * 32u + threadIdx.x;
    float s = 0.0f;
    if (j < cols)
#pragma unroll 8
        for (uint32_t b = threadIdx.y; b < blocks; b += kSumWarps)
            s += part[(static_cast<size_t>(b) * 3u + blockIdx.y) * cols + j];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || j >= cols) return;
#pragma unroll
    for (uint32_t k = 1; k < kSumWarps; ++k) s += sums[k][threadIdx.x];
    out[j] = from_f32<W>(s);
}

unsigned round_up(unsigned v, unsigned m) { return (v + m - 1u) / m * m; }

template <class T, class W, int V, int P>
void fwd_in_registers(const NormFwd &a, cudaStream_t s)
{
    const unsigned vectors = a.cols / V;
    if (vectors <= 32u * P) {
        const unsigned per = a.rows < 8 ? static_cast<unsigned>(a.rows) : 8u;
        norm_fwd_kernel<T, W, V, P, true>
            <<<static_cast<unsigned>((a.rows + per - 1) / per), dim3(32, per), 0, s>>>(a);
    } else {
        norm_fwd_kernel<T, W, V, P, false>
            <<<static_cast<unsigned>(a.rows), round_up((vectors + P - 1) / P, 32), 0, s>>>(a);
    }
    note_launch();
}

template <class T, class W>
void launch_column_sum(const NormBwd &a, const float *part, unsigned blocks, cudaStream_t s)
{
    column_sum_kernel<W><<<dim3((a.cols + 31u) / 32u, 3), dim3(32, kSumWarps), 0, s>>>(
        part, blocks, a.cols, static_cast<W *>(a.dgamma), static_cast<W *>(a.dbeta), static_cast<W *>(a.dbias));
    note_launch();
}

}  // namespace

template <class T>
cudaError_t stalled_waits_norm(uint64_t *count)
{
    return cudaMemcpyFromSymbol(count, g_stalled_waits, sizeof(uint64_t));
}

template <class T, class W>
cudaError_t launch_norm_fwd(const NormFwd &a, bool vectors, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(T);
    // Four vectors to a thread: the reductions' shuffles and the addresses cost a thread as much as ten of its elements
    // (16384 x 4096 in bf16: 92 us, 100 with two, 124 with one).  Up to 128 vectors, a warp holds a row, with no barrier.
    if (vectors && a.cols <= 32u * V) {
        fwd_in_registers<T, W, V, 1>(a, s);
    } else if (vectors && a.cols <= 64u * V) {
        fwd_in_registers<T, W, V, 2>(a, s);
    } else if (vectors && a.cols <= 4096u * V) {
        fwd_in_registers<T, W, V, 4>(a, s);
    } else if (!vectors && a.cols <= 4096u) {
        fwd_in_registers<T, W, 1, 4>(a, s);
    } else if (!vectors && a.cols <= 16384u) {
        fwd_in_registers<T, W, 1, 16>(a, s);
    } else {
        norm_fwd_long_kernel<T, W><<<static_cast<unsigned>(a.rows), 1024, 0, s>>>(a);
        note_launch();
    }
    return cudaGetLastError();
}

template <class T, class W>
cudaError_t launch_norm_bwd(const NormBwd &a, bool vectors, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(T);
    const NormBwdPlan plan = norm_bwd_plan(a.rows, a.cols);
    const bool weights = a.dgamma || a.dbeta || a.dbias;
    if (plan.fused) {
        unsigned blocks = plan.blocks;
        const dim3 block(plan.group, plan.per_block);
        const bool warp = plan.group == 32u;
        if (plan.blocks) {
            if (vectors && warp) {
                norm_bwd_kernel<T, W, V, true><<<plan.blocks, block, 0, s>>>(a);
            } else if (vectors) {
                blocks = plan.ring_blocks;
                const auto kernel = norm_bwd_ring_kernel<T, W, V>;
                static std::atomic<bool> done[16];
                if (const cudaError_t e = allow_shared(kernel, done)) return e;
                // the block's part of the SM's shared memory, and no more stages than rows
                const size_t stage = (a.dh.p ? 3u : 2u) * a.cols * sizeof(T), room = (226u * 1024u) / plan.ring_per_sm - 2048u;
                const size_t rows = (a.rows + blocks - 1) / blocks;
                size_t stages = room / stage < kRingStages ? room / stage : kRingStages;
                if (stages > rows) stages = rows;
                if (stages < 2) stages = 2;
                kernel<<<blocks, plan.ring_group, stages * stage, s>>>(a, static_cast<uint32_t>(stages));
            } else if (warp) {
                norm_bwd_kernel<T, W, 1, true><<<plan.blocks, block, 0, s>>>(a);
            } else {
                norm_bwd_kernel<T, W, 1, false><<<plan.blocks, block, 0, s>>>(a);
            }
            note_launch();
        }
        if (weights) launch_column_sum<T, W>(a, a.workspace, blocks, s);
    } else {
        if (plan.blocks) {
            norm_bwd_means_kernel<T, W><<<static_cast<unsigned>(a.rows), 1024, 0, s>>>(a);
            norm_bwd_columns_kernel<T, W><<<dim3((a.cols + 255u) / 256u, plan.blocks), 256, 0, s>>>(a);
            note_launch(), note_launch();
        }
        if (weights) launch_column_sum<T, W>(a, a.workspace + 2 * a.rows, plan.blocks, s);
    }
    return cudaGetLastError();
}

}  // namespace rngk
