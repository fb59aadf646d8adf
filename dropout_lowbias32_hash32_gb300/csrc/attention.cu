// attention.cu -- the extern "C" entry points of attention (include/rng.h):
// argument checks and the bucket boundaries.
#include "attention.h"
#include "layer_norm.h"

#include <cmath>
#include <cstring>

namespace rngk {
namespace {

// A whole number of up to 1024 bits, for the boundaries' exact comparison.
struct Big {
    uint32_t w[32] = {1};
    void mul(uint32_t m)
    {
        uint64_t carry = 0;
        for (uint32_t &x : w) {
            carry += static_cast<uint64_t>(x) * m;
            x = static_cast<uint32_t>(carry);
            carry >>= 32;
        }
    }
    bool operator>=(const Big &o) const
    {
        for (int i = 31; i >= 0; --i)
            if (w[i] != o.w[i]) return w[i] > o.w[i];
        return true;
    }
};

// The smallest n with n^m >= exact^(m - t) far^t, that is n >= exact (far /
// exact)^(t / m).  m <= 64 and far <= 2^10, so the powers stay below 2^641.
int32_t boundary(int32_t exact, int32_t far, int32_t m, int32_t t)
{
    const double v = exact * std::pow(static_cast<double>(far) / exact, static_cast<double>(t) / m);
    const double near = std::nearbyint(v);
    if (std::fabs(v - near) > 1e-6 * v) return static_cast<int32_t>(std::ceil(v));
    Big a, b;
    for (int32_t i = 0; i < m; ++i) {
        a.mul(static_cast<uint32_t>(near));
        b.mul(static_cast<uint32_t>(i < t ? far : exact));
    }
    return static_cast<int32_t>(near) + (a >= b ? 0 : 1);
}

}  // namespace

rng_status relative_buckets(const char *what, int32_t num_buckets, int32_t max_distance, bool bidirectional,
                            Buckets *out)
{
    if (num_buckets < (bidirectional ? 4 : 2) || num_buckets > kMaxBuckets || (bidirectional && num_buckets % 2))
        return fail(RNG_EINVAL, "%s: num_buckets = %d is outside %d .. %d%s", what, num_buckets, bidirectional ? 4 : 2,
                    kMaxBuckets, bidirectional ? " or odd" : "");
    const int32_t count = bidirectional ? num_buckets / 2 : num_buckets;
    const int32_t exact = count / 2, m = count - exact;
    if (max_distance <= exact || max_distance > kMaxDistance)
        return fail(RNG_EINVAL, "%s: max_distance = %d is outside %d .. %d", what, max_distance, exact + 1, kMaxDistance);
    out->total = num_buckets, out->count = count, out->past = bidirectional ? count : 0;
    out->max_distance = max_distance;
    for (int32_t i = 0; i < exact; ++i) out->starts[i] = i + 1;
    for (int32_t t = 1; t < m; ++t) out->starts[exact + t - 1] = boundary(exact, max_distance, m, t);
    return RNG_OK;
}

namespace {

struct Tensor {
    const char *name;
    const void *p;
    const int64_t *stride;
    int32_t len, heads;
    bool output;
};

// Bytes from a tensor's address to the end of its last element.
uint64_t extent(const rng_attention_args &a, const Tensor &t)
{
    return 2 * (static_cast<uint64_t>(a.batch - 1) * t.stride[0] + static_cast<uint64_t>(t.len - 1) * t.stride[1] +
                static_cast<uint64_t>(t.heads - 1) * t.stride[2] + a.head_dim);
}

bool empty(const rng_attention_args &a, const Tensor &t) { return a.batch == 0 || t.len == 0 || t.heads == 0; }

rng_status check_tensor(const char *what, const rng_attention_args &a, const Tensor &t)
{
    if (empty(a, t)) return RNG_OK;
    if (!t.p) return fail(RNG_EINVAL, "%s: %s is NULL", what, t.name);
    if (reinterpret_cast<uintptr_t>(t.p) % 16)
        return fail(RNG_EINVAL, "%s: %s is not on a 16-byte boundary", what, t.name);
    const int32_t n[3] = {a.batch, t.len, t.heads};
    double reach = a.head_dim;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (t.stride[i] <= 0 || t.stride[i] % 8 || t.stride[i] >= (int64_t(1) << 39))
            return fail(RNG_EINVAL, "%s: %s's stride %lld is not a positive multiple of 8 below 2^39", what, t.name,
                        static_cast<long long>(t.stride[i]));
        reach += static_cast<double>(n[i] - 1) * t.stride[i];
    }
    if (2 * reach > static_cast<double>(INT64_MAX) || extent(a, t) > UINTPTR_MAX - reinterpret_cast<uintptr_t>(t.p))
        return fail(RNG_EINVAL, "%s: %s runs past the end of the address space", what, t.name);
    if (t.output) {  // no element twice: from the smallest stride up, each clears what lies inside it
        int order[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (t.stride[order[j]] < t.stride[order[i]]) std::swap(order[i], order[j]);
        int64_t inside = a.head_dim;
        for (int i : order) {
            if (n[i] == 1) continue;
            if (t.stride[i] < inside) return fail(RNG_EINVAL, "%s: %s overlaps itself", what, t.name);
            inside += (n[i] - 1) * t.stride[i];
        }
    }
    return RNG_OK;
}

// Whether two tensors may share a byte.  Slices of one packed array (the same
// strides, one beside the other in each step of some stride) do not.
bool overlap(const rng_attention_args &a, const Tensor &x, const Tensor &y)
{
    if (empty(a, x) || empty(a, y)) return false;
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.p), y0 = reinterpret_cast<uintptr_t>(y.p);
    if (x0 + extent(a, x) <= y0 || y0 + extent(a, y) <= x0) return false;
    if (std::memcmp(x.stride, y.stride, 3 * sizeof(int64_t)) != 0) return true;
    for (int i = 0; i < 3; ++i) {
        const int64_t period = x.stride[i];
        if (period <= 0) continue;
        bool periodic = true;
        uint64_t fx = a.head_dim, fy = a.head_dim;  // elements used of one period
        for (int j = 0; j < 3; ++j) {
            if (j == i) continue;
            const int32_t nx = j == 0 ? a.batch : j == 1 ? x.len : x.heads, ny = j == 0 ? a.batch : j == 1 ? y.len : y.heads;
            if (x.stride[j] >= period) {
                periodic = periodic && x.stride[j] % period == 0;
            } else {
                fx += static_cast<uint64_t>(nx - 1) * x.stride[j];
                fy += static_cast<uint64_t>(ny - 1) * y.stride[j];
            }
        }
        const bool x_low = x0 <= y0;
        const uint64_t d = (x_low ? y0 - x0 : x0 - y0) / 2 % period;
        if (periodic && d >= (x_low ? fx : fy) && period - d >= (x_low ? fy : fx)) return false;
    }
    return true;
}

// A contiguous array beside the tensors; output: written.
struct Flat {
    const char *name;
    const void *p;
    uint64_t bytes;
    bool output;
};

// A tensor's dimensions from the largest stride to the smallest, in bytes, and
// what one entry of the dimensions before reaches.
struct Nest {
    int32_t n[3];
    uint64_t step[3], reach[4];
};

Nest nest_of(const rng_attention_args &a, const Tensor &t)
{
    const int32_t n[3] = {a.batch, t.len, t.heads};
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (t.stride[order[j]] > t.stride[order[i]]) std::swap(order[i], order[j]);
    Nest x;
    x.reach[3] = 2 * static_cast<uint64_t>(a.head_dim);
    for (int k = 2; k >= 0; --k) {
        x.n[k] = n[order[k]], x.step[k] = 2 * static_cast<uint64_t>(t.stride[order[k]]);
        x.reach[k] = x.reach[k + 1] + (x.n[k] - 1) * x.step[k];
    }
    return x;
}

// Whether [f0, f1) shares a byte with the tensor's part at `at` of the
// dimensions from k on: with its first or its last entry there, or it holds one
// between them.  Entries that overlap each other (an input's may) count as
// without gaps.
bool meets(const Nest &x, int k, uintptr_t at, uintptr_t f0, uintptr_t f1)
{
    if (f1 <= at || at + x.reach[k] <= f0) return false;
    if (k == 3) return true;
    if (x.n[k] == 1) return meets(x, k + 1, at, f0, f1);
    const uint64_t step = x.step[k], inside = x.reach[k + 1], last = x.n[k] - 1;
    if (step < inside) return true;
    const uint64_t first = f0 < at + inside ? 0 : (f0 - at - inside) / step + 1, end = (f1 - 1 - at) / step;
    const uint64_t to = end < last ? end : last;
    if (first > to) return false;
    return to - first > 1 || meets(x, k + 1, at + first * step, f0, f1) || meets(x, k + 1, at + to * step, f0, f1);
}

// Outputs share no byte with anything else (the tensors among themselves are
// check_tensors's).
template <size_t N, size_t M>
rng_status check_flat(const char *what, const rng_attention_args &a, const Flat (&f)[M], const Tensor (&t)[N])
{
    for (size_t i = 0; i < M; ++i) {
        if (!f[i].p || f[i].bytes == 0) continue;
        const uintptr_t f0 = reinterpret_cast<uintptr_t>(f[i].p), f1 = f0 + f[i].bytes;
        if (f1 < f0) return fail(RNG_EINVAL, "%s: %s runs past the end of the address space", what, f[i].name);
        for (const Tensor &x : t) {
            const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.p);
            if (!(x.output || f[i].output) || empty(a, x) || f1 <= x0 || x0 + extent(a, x) <= f0) continue;
            if (meets(nest_of(a, x), 0, x0, f0, f1))
                return fail(RNG_EINVAL, "%s: %s and %s overlap", what, x.name, f[i].name);
        }
        for (size_t j = 0; j < i; ++j) {
            const uintptr_t other = reinterpret_cast<uintptr_t>(f[j].p);
            if (f[j].p && (f[i].output || f[j].output) && f0 < other + f[j].bytes && other < f1)
                return fail(RNG_EINVAL, "%s: %s and %s overlap", what, f[j].name, f[i].name);
        }
    }
    return RNG_OK;
}

// Bytes of lse, and of the table or its gradient.
uint64_t lse_bytes(const Attention &t) { return uint64_t(4) * t.batch * t.heads * t.len_q; }
uint64_t table_bytes(const Attention &t) { return uint64_t(2) * t.buckets.total * t.heads; }

// The sizes and options, without the pointers.
rng_status make(const char *what, const rng_attention_args *args, bool sizes_only, Attention *out)
{
    if (!args) return fail(RNG_EINVAL, "%s: args is NULL", what);
    const rng_attention_args &a = *args;
    if (a.dtype != RNG_F16 && a.dtype != RNG_BF16)
        return fail(RNG_EINVAL, "%s: dtype %d is neither RNG_F16 nor RNG_BF16", what, a.dtype);
    if (a.batch < 0 || a.len_q < 0 || a.len_k < 0 || a.heads_q < 0 || a.heads_kv < 0)
        return fail(RNG_EINVAL, "%s: a size is negative", what);
    if (a.head_dim < 8 || a.head_dim > 128 || a.head_dim % 8)
        return fail(RNG_EINVAL, "%s: head_dim = %d is not a multiple of 8 in 8 .. 128", what, a.head_dim);
    if (a.heads_q && (a.heads_kv == 0 || a.heads_q % a.heads_kv))
        return fail(RNG_EINVAL, "%s: heads_q = %d is not a multiple of heads_kv = %d", what, a.heads_q, a.heads_kv);
    if (static_cast<int64_t>(a.batch) * a.heads_q > 0x7FFFFFFF / 2)
        return fail(RNG_EINVAL, "%s: batch * heads_q exceeds 2^30", what);
    if (a.len_q > (1 << 30) || a.len_k > (1 << 30)) return fail(RNG_EINVAL, "%s: a length exceeds 2^30", what);
    Attention &t = *out;
    t = Attention{};
    t.batch = a.batch, t.len_q = a.len_q, t.len_k = a.len_k, t.heads = a.heads_q, t.heads_kv = a.heads_kv;
    t.dim = a.head_dim, t.group = a.heads_kv ? a.heads_q / a.heads_kv : 1;
    t.causal = a.causal != 0, t.last = a.queries_last != 0;
    t.table = a.bias_table, t.dtable = a.dbias_table, t.scale = a.scale;
    if (a.bias_table || a.dbias_table) {
        if (rng_status st = relative_buckets(what, a.num_buckets, a.max_distance, a.bidirectional != 0, &t.buckets))
            return st;
        if (a.dbias_table && !a.bias_table)
            return fail(RNG_EINVAL, "%s: dbias_table without a bias_table", what);
    }
    if (sizes_only) return RNG_OK;
    if (!(a.p >= 0.0f && a.p < 1.0f)) return fail(RNG_EINVAL, "%s: p = %g is outside [0, 1)", what, (double)a.p);
    if (!std::isfinite(a.scale)) return fail(RNG_EINVAL, "%s: scale is not finite", what);
    const struct {
        const char *name;
        const void *p;
        size_t size;
    } small[] = {{"lse", a.lse, 4}, {"key_lengths", a.key_lengths, 4}, {"bias_table", a.bias_table, 2},
                 {"dbias_table", a.dbias_table, 2}};
    for (const auto &x : small)
        if (reinterpret_cast<uintptr_t>(x.p) % x.size)
            return fail(RNG_EINVAL, "%s: %s is not aligned to its %zu-byte element", what, x.name, x.size);
    auto strides = [](const int64_t *s) { return Strides{s[0], s[1], s[2]}; };
    t.q = a.q, t.k = a.k, t.v = a.v, t.lse = a.lse, t.key_lengths = a.key_lengths;
    t.qs = strides(a.q_stride), t.ks = strides(a.k_stride), t.vs = strides(a.v_stride), t.os = strides(a.o_stride);
    t.mask = make_mask(a.p, a.seed);
    t.first = a.first_counter;
    t.workspace = a.workspace;
    return RNG_OK;
}

template <size_t N>
rng_status check_tensors(const char *what, const rng_attention_args &a, const Tensor (&t)[N])
{
    for (const Tensor &x : t)
        if (rng_status st = check_tensor(what, a, x)) return st;
    for (size_t i = 0; i < N; ++i)
        for (size_t j = 0; j < N; ++j)
            if (t[i].output && j != i && (!t[j].output || j < i) && overlap(a, t[i], t[j]))
                return fail(RNG_EINVAL, "%s: %s and %s overlap", what, t[i].name, t[j].name);
    return RNG_OK;
}

rng_status check_workspace(const char *what, const rng_attention_args &a, size_t need)
{
    if (need && (!a.workspace || reinterpret_cast<uintptr_t>(a.workspace) % 16 || a.workspace_bytes < need))
        return fail(RNG_EINVAL, "%s: workspace of %zu bytes at a 16-byte boundary wanted, %zu given", what, need,
                    a.workspace ? a.workspace_bytes : size_t(0));
    return RNG_OK;
}

}  // namespace
}  // namespace rngk

using namespace rngk;

extern "C" {

rng_status rng_relative_bucket(int64_t relative_position, int32_t num_buckets, int32_t max_distance,
                               int32_t bidirectional, int32_t *bucket)
{
    if (!bucket) return fail(RNG_EINVAL, "rng_relative_bucket: bucket is NULL");
    Buckets b{};
    if (rng_status st = relative_buckets("rng_relative_bucket", num_buckets, max_distance, bidirectional != 0, &b))
        return st;
    // as far out as any distance reaches (and -INT64_MIN has no value)
    const int64_t far = kMaxDistance + 1;
    *bucket = bucket_of(b, relative_position > far ? far : relative_position < -far ? -far : relative_position);
    return RNG_OK;
}

size_t rng_attention_fwd_workspace(const rng_attention_args *args)
{
    Attention t;
    return make("rng_attention_fwd_workspace", args, true, &t) == RNG_OK ? attention_fwd_workspace(t) : 0;
}

size_t rng_attention_bwd_workspace(const rng_attention_args *args)
{
    Attention t;
    return make("rng_attention_bwd_workspace", args, true, &t) == RNG_OK ? attention_bwd_workspace(t) : 0;
}

rng_status rng_attention_fwd(const rng_attention_args *args, void *stream)
{
    static const char what[] = "rng_attention_fwd";
    Attention t;
    if (rng_status st = make(what, args, false, &t)) return st;
    const rng_attention_args &a = *args;
    if (t.batch == 0 || t.len_q == 0 || t.heads == 0) return RNG_OK;
    const Tensor tensors[] = {{"q", a.q, a.q_stride, a.len_q, a.heads_q, false},
                              {"k", a.k, a.k_stride, a.len_k, a.heads_kv, false},
                              {"v", a.v, a.v_stride, a.len_k, a.heads_kv, false},
                              {"o", a.o, a.o_stride, a.len_q, a.heads_q, true}};
    if (rng_status st = check_tensors(what, a, tensors)) return st;
    const size_t need = attention_fwd_workspace(t);
    if (rng_status st = check_workspace(what, a, need)) return st;
    const Flat flat[] = {{"key_lengths", a.key_lengths, uint64_t(4) * t.batch, false},
                         {"bias_table", a.bias_table, table_bytes(t), false},
                         {"lse", a.lse, lse_bytes(t), true},
                         {"workspace", a.workspace, need, true}};
    if (rng_status st = check_flat(what, a, flat, tensors)) return st;
    t.out = a.o;
    clear_error();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a.dtype == RNG_F16 ? launch_attention_fwd<__half>(t, s) : launch_attention_fwd<__nv_bfloat16>(t, s);
    return e == cudaSuccess ? RNG_OK : cuda_fail(e, what);
}

rng_status rng_attention_bwd(const rng_attention_args *args, void *stream)
{
    static const char what[] = "rng_attention_bwd";
    Attention t;
    if (rng_status st = make(what, args, false, &t)) return st;
    const rng_attention_args &a = *args;
    if (t.batch == 0 && !t.dtable) return RNG_OK;
    const Tensor tensors[] = {{"q", a.q, a.q_stride, a.len_q, a.heads_q, false},
                              {"k", a.k, a.k_stride, a.len_k, a.heads_kv, false},
                              {"v", a.v, a.v_stride, a.len_k, a.heads_kv, false},
                              {"o", a.o, a.o_stride, a.len_q, a.heads_q, false},
                              {"d_o", a.d_o, a.do_stride, a.len_q, a.heads_q, false},
                              {"dq", a.dq, a.dq_stride, a.len_q, a.heads_q, true},
                              {"dk", a.dk, a.dk_stride, a.len_k, a.heads_kv, true},
                              {"dv", a.dv, a.dv_stride, a.len_k, a.heads_kv, true}};
    if (rng_status st = check_tensors(what, a, tensors)) return st;
    if (!a.lse && t.batch && t.len_q && t.heads) return fail(RNG_EINVAL, "%s: lse is NULL", what);
    const size_t need = attention_bwd_workspace(t);
    if (rng_status st = check_workspace(what, a, need)) return st;
    const Flat flat[] = {{"key_lengths", a.key_lengths, uint64_t(4) * t.batch, false},
                         {"bias_table", a.bias_table, table_bytes(t), false},
                         {"lse", a.lse, lse_bytes(t), false},
                         {"dbias_table", a.dbias_table, table_bytes(t), true},
                         {"workspace", a.workspace, need, true}};
    if (rng_status st = check_flat(what, a, flat, tensors)) return st;
    t.o = a.o, t.d_o = a.d_o, t.dq = a.dq, t.dk = a.dk, t.dv = a.dv;
    auto strides = [](const int64_t *s) { return Strides{s[0], s[1], s[2]}; };
    t.dos = strides(a.do_stride), t.dqs = strides(a.dq_stride), t.dks = strides(a.dk_stride), t.dvs = strides(a.dv_stride);
    clear_error();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a.dtype == RNG_F16 ? launch_attention_bwd<__half>(t, s) : launch_attention_bwd<__nv_bfloat16>(t, s);
    return e == cudaSuccess ? RNG_OK : cuda_fail(e, what);
}

rng_status rng_debug_stalled_waits(uint64_t *count)
{
    if (!count) return fail(RNG_EINVAL, "rng_debug_stalled_waits: count is NULL");
    clear_error();
    cudaError_t (*const kernels[])(uint64_t *) = {stalled_waits_fwd, stalled_waits_bwd, stalled_waits_norm<float>,
                                                  stalled_waits_norm<__half>, stalled_waits_norm<__nv_bfloat16>};
    *count = 0;
    cudaError_t e = cudaSuccess;
    for (const auto kernel : kernels) {
        uint64_t n = 0;
        if (e == cudaSuccess) e = kernel(&n);
        *count += n;
    }
    return e == cudaSuccess ? RNG_OK : cuda_fail(e, "rng_debug_stalled_waits");
}

}  // extern "C"
