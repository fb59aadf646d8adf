// attention_bwd.cu -- attention backward (include/rng.h, rng_attention_bwd): one warp to a query (or key),
// 32 keys (queries) at a time, a lane to each for the scores and a lane to
// every 32nd column of the head dimension for the products.
#include "attention.h"

namespace rngk {
namespace {

constexpr int kCols = 4;  // columns of a head (up to 128) in a lane

struct Place {
    int32_t b, a, i;  // batch, head, position
};

__device__ __forceinline__ Place place_of(int64_t row, int32_t heads, int32_t len)
{
    const int64_t ba = row / len;
    return Place{static_cast<int32_t>(ba / heads), static_cast<int32_t>(ba % heads), static_cast<int32_t>(row % len)};
}

template <class T>
__device__ __forceinline__ const T *at(const void *p, const Strides &s, int64_t b, int64_t l, int64_t h)
{
    return static_cast<const T *>(p) + b * s.batch + l * s.len + h * s.head;
}

template <class T>
__device__ float dot(const T *x, const T *y, int32_t n)
{
    float s = 0.0f;
    for (int32_t d = 0; d < n; ++d) s += to_f32(x[d]) * to_f32(y[d]);
    return s;
}

template <class T>
__device__ __forceinline__ void add_row(float (&acc)[kCols], float w, const T *row, int32_t dim, uint32_t lane)
{
#pragma unroll
    for (int k = 0; k < kCols; ++k)
        if (lane + 32 * k < dim) acc[k] += w * to_f32(row[lane + 32 * k]);
}

template <class T>
__device__ __forceinline__ void put_row(T *row, const float (&acc)[kCols], float w, int32_t dim, uint32_t lane)
{
#pragma unroll
    for (int k = 0; k < kCols; ++k)
        if (lane + 32 * k < dim) row[lane + 32 * k] = from_f32<T>(acc[k] * w);
}

__device__ __forceinline__ float warp_sum(float v)
{
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    return v;
}
// The score of a visible pair.
template <class T>
__device__ float score(const Attention &a, const T *q, const T *k, int32_t head, int32_t rel)
{
    float s = dot(q, k, a.dim) * a.scale;
    if (a.table) s += to_f32(static_cast<const T *>(a.table)[bucket_of(a.buckets, rel) * a.heads + head]);
    return s;
}

__device__ __forceinline__ uint32_t counter(const Attention &a, const Place &x, uint32_t j)
{
    return a.first + ((static_cast<uint32_t>(x.b) * a.heads + x.a) * a.len_q + x.i) * static_cast<uint32_t>(a.len_k) + j;
}

// Workspace of the backward pass: delta of every query, then each query's
// sums of dS by bucket.
__host__ __device__ __forceinline__ int64_t queries(const Attention &a)
{
    return static_cast<int64_t>(a.batch) * a.heads * a.len_q;
}

// The probability of a visible pair and its dS.
template <class T>
__device__ __forceinline__ void gradient(const Attention &a, const T *q, const T *k, const T *v, const T *d_o, float lse,
                                         float delta, const Place &x, int32_t j, int32_t pos, float &kept, float &ds)
{
    // a query that sees no key, or only scores of -inf, has lse = -inf
    const float p = lse == -INFINITY ? 0.0f : __expf(score(a, q, k, x.a, j - pos) - lse);
    float dp = dot(d_o, v, a.dim);
    kept = p;
    if (a.mask.threshold) {
        const float keep = keeps(a.mask, counter(a, x, j)) ? a.mask.scale : 0.0f;
        kept *= keep, dp *= keep;
    }
    ds = p * (dp - delta);
}

template <class T>
__global__ void __launch_bounds__(128) dq_kernel(const __grid_constant__ Attention a)
{
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.y;
    if (row >= queries(a)) return;
    const uint32_t lane = threadIdx.x;
    const Place x = place_of(row, a.heads, a.len_q);
    const int32_t keys = keys_of(a, x.b), pos = first_position(a, keys) + x.i, hk = x.a / a.group;
    const int32_t end = a.causal && pos + 1 < keys ? pos + 1 : keys;
    const T *q = at<T>(a.q, a.qs, x.b, x.i, x.a), *o = at<T>(a.o, a.os, x.b, x.i, x.a);
    const T *d_o = at<T>(a.d_o, a.dos, x.b, x.i, x.a);
    float *ws = static_cast<float *>(a.workspace);
    float delta = 0.0f, lse = a.lse[row], acc[kCols] = {}, by_bucket[kMaxBuckets / 32] = {};
    for (int32_t d = lane; d < a.dim; d += 32) delta += to_f32(o[d]) * to_f32(d_o[d]);
    delta = warp_sum(delta);
    if (lane == 0) ws[row] = delta;
    for (int32_t j0 = 0; j0 < end; j0 += 32) {
        const int32_t j = j0 + lane;
        float kept, ds = 0.0f;
        if (j < end)
            gradient(a, q, at<T>(a.k, a.ks, x.b, j, hk), at<T>(a.v, a.vs, x.b, j, hk), d_o, lse, delta, x, j, pos, kept, ds);
        const int32_t bucket = a.dtable ? bucket_of(a.buckets, j - pos) : 0;
        for (int k = 0; k < 32 && j0 + k < end; ++k) {
            const float w = __shfl_sync(0xFFFFFFFFu, ds, k);
            add_row(acc, w, at<T>(a.k, a.ks, x.b, j0 + k, hk), a.dim, lane);
            const uint32_t n = __shfl_sync(0xFFFFFFFFu, bucket, k);
#pragma unroll
            for (uint32_t m = 0; m < kMaxBuckets / 32; ++m)
                if (n == lane + 32 * m) by_bucket[m] += w;
        }
    }
    put_row(static_cast<T *>(a.dq) + x.b * a.dqs.batch + x.i * a.dqs.len + x.a * a.dqs.head, acc, a.scale, a.dim, lane);
    if (a.dtable)
        for (uint32_t m = 0; m < kMaxBuckets / 32; ++m)
            if (lane + 32 * m < a.buckets.total)
                ws[queries(a) + row * a.buckets.total + lane + 32 * m] = by_bucket[m];
}

template <class T>
__global__ void __launch_bounds__(128) dkv_kernel(const __grid_constant__ Attention a)
{
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.y;
    if (row >= static_cast<int64_t>(a.batch) * a.heads_kv * a.len_k) return;
    const uint32_t lane = threadIdx.x;
    const Place y = place_of(row, a.heads_kv, a.len_k);
    const int32_t keys = keys_of(a, y.b), pos0 = first_position(a, keys), j = y.i;
    const T *k = at<T>(a.k, a.ks, y.b, j, y.a), *v = at<T>(a.v, a.vs, y.b, j, y.a);
    const float *ws = static_cast<const float *>(a.workspace);
    float dk[kCols] = {}, dv[kCols] = {};
    int32_t begin = a.causal && j > pos0 ? j - pos0 : 0;  // the first query that sees key j
    if (j >= keys) begin = a.len_q;
    for (int32_t h = y.a * a.group; h < (y.a + 1) * a.group; ++h) {
        for (int32_t i0 = begin; i0 < a.len_q; i0 += 32) {
            const int32_t i = i0 + lane;
            const Place x{y.b, h, i};
            float kept = 0.0f, ds = 0.0f;
            if (i < a.len_q) {
                const int64_t r = (static_cast<int64_t>(y.b) * a.heads + h) * a.len_q + i;
                gradient(a, at<T>(a.q, a.qs, y.b, i, h), k, v, at<T>(a.d_o, a.dos, y.b, i, h), a.lse[r], ws[r], x, j,
                         pos0 + i, kept, ds);
            }
            for (int n = 0; n < 32 && i0 + n < a.len_q; ++n) {
                add_row(dk, __shfl_sync(0xFFFFFFFFu, ds, n), at<T>(a.q, a.qs, y.b, i0 + n, h), a.dim, lane);
                add_row(dv, __shfl_sync(0xFFFFFFFFu, kept, n), at<T>(a.d_o, a.dos, y.b, i0 + n, h), a.dim, lane);
            }
        }
    }
    put_row(static_cast<T *>(a.dk) + y.b * a.dks.batch + j * a.dks.len + y.a * a.dks.head, dk, a.scale, a.dim, lane);
    put_row(static_cast<T *>(a.dv) + y.b * a.dvs.batch + j * a.dvs.len + y.a * a.dvs.head, dv, 1.0f, a.dim, lane);
}

// dtable[n, head] from every query's sums: a block to each, its threads' sums
// added in a fixed order.
template <class T>
__global__ void __launch_bounds__(256) dtable_kernel(const __grid_constant__ Attention a)
{
    __shared__ float sums[8];
    const int32_t n = blockIdx.x, head = blockIdx.y;
    const float *ws = static_cast<const float *>(a.workspace) + queries(a);
    float s = 0.0f;
    for (int64_t r = threadIdx.x; r < static_cast<int64_t>(a.batch) * a.len_q; r += 256)
        s += ws[((r / a.len_q * a.heads + head) * a.len_q + r % a.len_q) * a.buckets.total + n];
    s = warp_sum(s);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) s += sums[w];
        static_cast<T *>(a.dtable)[n * a.heads + head] = from_f32<T>(s);
    }
}

}  // namespace

size_t attention_bwd_workspace(const Attention &a)
{
    return static_cast<size_t>(queries(a)) * (1 + (a.dtable ? a.buckets.total : 0)) * sizeof(float);
}

template <class T>
cudaError_t launch_attention_bwd(const Attention &a, cudaStream_t s)
{
    const int64_t nq = queries(a), nk = static_cast<int64_t>(a.batch) * a.heads_kv * a.len_k;
    if (nq) {
        dq_kernel<T><<<static_cast<unsigned>((nq + 3) / 4), dim3(32, 4), 0, s>>>(a);
        note_launch();
    }
    if (nk) {
        dkv_kernel<T><<<static_cast<unsigned>((nk + 3) / 4), dim3(32, 4), 0, s>>>(a);
        note_launch();
    }
    if (a.dtable && a.heads) {
        dtable_kernel<T><<<dim3(a.buckets.total, a.heads), 256, 0, s>>>(a);
        note_launch();
    }
    return cudaGetLastError();
}

template cudaError_t launch_attention_bwd<__half>(const Attention &, cudaStream_t);
template cudaError_t launch_attention_bwd<__nv_bfloat16>(const Attention &, cudaStream_t);

}  // namespace rngk
