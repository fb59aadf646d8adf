// attention.h -- what the attention kernels are launched with (host side of
// attention.cu), and the device helpers that every one of them shares: the
// position of a query, the mask, the buckets.
#pragma once

#include "element.cuh"
#include "internal.h"

namespace rngk {

constexpr int kMaxBuckets = 128;
constexpr int kMaxDistance = 1024;

// One direction's buckets by the distances at which bucket 1, 2, ... begin
// (count - 1 of them, ascending); `past` is added for keys past the query.
struct Buckets {
    int32_t total, count, past, max_distance;
    int32_t starts[kMaxBuckets];
};

// Division by a number that a launch fixes: a product's high half and a shift
// (the multiplier rounded up is exact for dividends below 2^31).  The kernels
// cut an item's index with it, which their roles all wait for.
struct Divider {
    uint32_t by, multiplier, shift;
    Divider() = default;
    explicit Divider(uint32_t d) : by(d), multiplier(0), shift(0)
    {
        if (d < 2) return;
        uint32_t log = 1;
        while ((uint64_t(1) << log) < d) ++log;
        multiplier = static_cast<uint32_t>(((uint64_t(1) << (31 + log)) + d - 1) / d);
        shift = log - 1;
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return by < 2 ? n : __umulhi(n, multiplier) >> shift; }
    __device__ __forceinline__ void divide(uint32_t n, int32_t &q, int32_t &r) const
    {
        q = static_cast<int32_t>(quotient(n));
        r = static_cast<int32_t>(n) - q * static_cast<int32_t>(by);
    }
};

struct Strides {
    int64_t batch, len, head;
};

struct Attention {
    int32_t batch, len_q, len_k, heads, heads_kv, dim, group;
    const void *q, *k, *v, *o, *d_o;
    void *out, *dq, *dk, *dv;
    Strides qs, ks, vs, os, dos, dqs, dks, dvs;
    float *lse;
    const int32_t *key_lengths;
    bool causal, last;
    float scale;
    const void *table;
    void *dtable;
    Buckets buckets;
    Mask mask;
    uint32_t first;
    void *workspace;
};

// Attention of a tree of tokens over a cache: len_q nodes, key_lengths the rows cached before them.
struct TreeAttention {
    Attention a;
    const int32_t *parents;
};

// The move of accepted tokens' rows in caches of the same sizes and strides.
struct CacheKeep {
    int32_t batch, nodes, len_k, heads, dim;
    Strides strides;
    const int32_t *lengths, *path, *accepted;
    int32_t *new_lengths;
};
cudaError_t launch_cache_keep(const CacheKeep &c, void *const *caches, int32_t count, cudaStream_t s);

rng_status relative_buckets(const char *what, int32_t num_buckets, int32_t max_distance, bool bidirectional,
                            Buckets *out);

// Waits that ran out in the forward, the backward and the tree's kernels, on the current device.
cudaError_t stalled_waits_fwd(uint64_t *count);
cudaError_t stalled_waits_bwd(uint64_t *count);
cudaError_t stalled_waits_tree(uint64_t *count);

size_t attention_fwd_workspace(const Attention &a);
size_t attention_bwd_workspace(const Attention &a);
template <class T>
cudaError_t launch_attention_fwd(const Attention &a, cudaStream_t s);
template <class T>
cudaError_t launch_attention_bwd(const Attention &a, cudaStream_t s);
size_t tree_attention_workspace(const TreeAttention &t);
template <class T>
cudaError_t launch_tree_attention(const TreeAttention &t, cudaStream_t s);

__host__ __device__ __forceinline__ int32_t bucket_of(const Buckets &b, int64_t rel)
{
    int64_t d = rel > 0 ? (b.past ? rel : 0) : -rel;
    if (d > b.max_distance) d = b.max_distance;
    int lo = 0, hi = b.count - 1;  // the number of starts at or below d
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (b.starts[mid] <= d) lo = mid + 1;
        else hi = mid;
    }
    return lo + (rel > 0 ? b.past : 0);
}

// The number of keys of a batch entry, and the position of its query 0.
__device__ __forceinline__ int32_t keys_of(const Attention &a, int32_t b)
{
    if (!a.key_lengths) return a.len_k;
    const int32_t n = a.key_lengths[b];
    return n < 0 ? 0 : n > a.len_k ? a.len_k : n;
}
__device__ __forceinline__ int32_t first_position(const Attention &a, int32_t keys) { return a.last ? keys - a.len_q : 0; }

// The bias by relative position is tabulated for -reach .. reach - 1.  A piece of
// 32 queries by 64 keys (backward: 32 by 32) has 95 positions; one that is not
// past the last bucket's start as a whole reaches at most 94 past it.
__host__ __device__ __forceinline__ int32_t bias_reach(const Buckets &b) { return b.max_distance + 160; }

// Whether the forward kernels with a bias are needed: those without take the
// maximum before the scores are scaled, and so want a scale above 0.
inline bool has_bias(const Attention &a) { return a.table != nullptr || !(a.scale > 0.0f); }

// Whether P and dS enter the products that follow as two 16-bit terms, the
// rounded value and what rounding left.  One rounding adds an error as large as
// the output's own: 1.4 of it together over many pairs, but up to 1.7 over few,
// where chance decides.  The rule looks at a single batch entry, so that what a
// request is batched with does not change its rounding.  So few pairs alone are
// bound by latency (a token of 8 heads, 301 keys: 8.9 us, 8.6 with one term); in
// large batches the second term costs (512 entries of 60 x 60 positions, 8 heads,
// p = 0.1: forward 105 and 99 us, backward 160 and 136; 256 of 180 x 180, 2 heads:
// 33 and 30 forward; 16 tokens of 16 heads, 4096 keys, the bound: 45 and 38), and above the bound it would cost
// as much at any size.
inline bool two_terms(const Attention &a) { return static_cast<int64_t>(a.len_q) * a.len_k * a.heads <= 65536; }

inline int32_t log2_of(int32_t power)
{
    int32_t n = 0;
    while ((1 << n) < power) ++n;
    return n;
}

// Heads of one key head that lie side by side in a tile of 128 rows, so that
// they read its keys once: all of them, where a tile is a whole number of
// them and no head has a bias of its own.  At least 1, also without query heads.
inline int32_t packed_heads(const Attention &a)
{
    return !has_bias(a) && a.group >= 1 && a.group <= 64 && (a.group & (a.group - 1)) == 0 ? a.group : 1;
}

}  // namespace rngk
