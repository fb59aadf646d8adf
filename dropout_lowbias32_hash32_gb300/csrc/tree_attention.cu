// tree_attention.cu -- attention of a tree of drafted tokens over a cache
// (include/rng.h, rng_tree_attention_fwd).
//
// A block to a node, a head and a batch entry: scores of 128 keys at a time, a
// key to a thread, with the running maximum and sum of the softmax.
#include "attention.h"

namespace rngk {
namespace {

constexpr int kThreads = 128, kMaxNodes = RNG_MAX_TREE_NODES;

template <class T>
__global__ void __launch_bounds__(kThreads) tree_attention_kernel(const __grid_constant__ TreeAttention p)
{
    __shared__ float q[128], weight[kThreads], part[4];
    __shared__ int16_t depth_of[kMaxNodes];  // of the nodes of the line, -1 for the others
    __shared__ int32_t line;                 // the line's length, 0 for none
    const Attention &a = p.a;
    const int32_t i = blockIdx.x % a.len_q, rest = blockIdx.x / a.len_q, h = rest % a.heads, b = rest / a.heads;
    const int32_t room = a.len_k - a.len_q;
    const int32_t cached = a.key_lengths ? min(max(a.key_lengths[b], 0), room) : room;
    const uint32_t x = threadIdx.x;
    if (x < kMaxNodes) depth_of[x] = -1;
    if (x < a.dim) q[x] = to_f32(static_cast<const T *>(a.q)[b * a.qs.batch + i * a.qs.len + h * a.qs.head + x]);
    __syncthreads();
    if (x == 0) {
        const int32_t *parents = p.parents ? p.parents + static_cast<int64_t>(b) * a.len_q : nullptr;
        int32_t n = 0, at = i;
        for (; at >= 0; ++n) {
            depth_of[at] = static_cast<int16_t>(n);
            const int32_t up = parents ? parents[at] : at - 1;
            if (up < -1 || up >= at) {
                n = -1;  // absent
                break;
            }
            at = up;
        }
        line = n < 0 ? 0 : n;
        for (int32_t t = 0; t <= i; ++t)
            if (depth_of[t] >= 0) depth_of[t] = static_cast<int16_t>(n - 1 - depth_of[t]);
    }
    __syncthreads();
    const int32_t keys = line ? cached + a.len_q : 0, pos = cached + line - 1;
    const T *k = static_cast<const T *>(a.k) + b * a.ks.batch + h / a.group * a.ks.head;
    const T *v = static_cast<const T *>(a.v) + b * a.vs.batch + h / a.group * a.vs.head;
    float top = -INFINITY, sum = 0.0f, o = 0.0f;
    auto over_block = [&](float y, bool largest) {
#pragma unroll
        for (int d = 16; d; d /= 2) {
            const float z = __shfl_xor_sync(0xFFFFFFFFu, y, d);
            y = largest ? fmaxf(y, z) : y + z;
        }
        __syncthreads();
        if (x % 32 == 0) part[x / 32] = y;
        __syncthreads();
        return largest ? fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])) : part[0] + part[1] + part[2] + part[3];
    };
    for (int32_t j0 = 0; j0 < keys; j0 += kThreads) {
        const int32_t j = j0 + static_cast<int32_t>(x), node = j - cached;
        float s = -INFINITY;
        if (j < keys && (node < 0 || depth_of[node] >= 0)) {
            float dot = 0.0f;
            for (int32_t d = 0; d < a.dim; ++d) dot += q[d] * to_f32(k[j * a.ks.len + d]);
            s = dot * a.scale;
            if (a.table)
                s += to_f32(static_cast<const T *>(a.table)[bucket_of(a.buckets, (node < 0 ? j : cached + depth_of[node]) - pos) * a.heads + h]);
        }
        const float next = fmaxf(top, over_block(s, true));
        const float e = s == -INFINITY ? 0.0f : exp2f((s - next) * 1.4426950408889634f);
        const float fade = top == -INFINITY ? 0.0f : exp2f((top - next) * 1.4426950408889634f);
        top = next;
        sum = sum * fade + over_block(e, false);
        weight[x] = e;
        __syncthreads();
        o *= fade;
        if (x < a.dim)
            for (int32_t t = 0; t < kThreads && j0 + t < keys; ++t)
                if (weight[t] > 0.0f) o += weight[t] * to_f32(v[(j0 + t) * a.vs.len + x]);
        __syncthreads();
    }
    if (x < a.dim)
        static_cast<T *>(a.out)[b * a.os.batch + i * a.os.len + h * a.os.head + x] = from_f32<T>(sum == 0.0f ? 0.0f : o / sum);
    if (a.lse && x == 0)
        a.lse[(static_cast<int64_t>(b) * a.heads + h) * a.len_q + i] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t stalled_waits_tree(uint64_t *count)
{
    *count = 0;  // no waits
    return cudaSuccess;
}

size_t tree_attention_workspace(const TreeAttention &) { return 0; }

template <class T>
cudaError_t launch_tree_attention(const TreeAttention &t, cudaStream_t s)
{
    const int64_t blocks = static_cast<int64_t>(t.a.batch) * t.a.heads * t.a.len_q;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    tree_attention_kernel<T><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(t);
    note_launch();
    return cudaGetLastError();
}

template cudaError_t launch_tree_attention<__half>(const TreeAttention &, cudaStream_t);
template cudaError_t launch_tree_attention<__nv_bfloat16>(const TreeAttention &, cudaStream_t);

}  // namespace rngk
