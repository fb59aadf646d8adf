// layer_norm.cu -- the extern "C" entry points of bias + dropout + residual +
// layer norm (include/rng.h): argument checks, the choice between 16-byte and
// single-element accesses, the backward pass's plan.
#include "layer_norm.h"

#include <cmath>

namespace rngk {

// The fused kernel holds 8 elements a thread, 1024 threads to an SM (64
// registers each), the one with a ring 16, 512 to an SM (128 registers): both up
// to 8192 columns.  Every block writes a row of partial sums, so few rows are
// not spread over all blocks: two to a block, where that still gives every SM
// one.  For longer rows, chunks of rows such that about 8 blocks of 256 columns
// an SM run.
NormBwdPlan norm_bwd_plan(size_t rows, size_t cols)
{
    NormBwdPlan p{};
    const size_t sms = sm_count();
    auto spread = [&](size_t groups, size_t per_sm) {  // blocks for that many groups of rows
        const size_t blocks = groups / 2 > sms ? groups / 2 : groups < sms ? groups : sms;
        return static_cast<unsigned>(blocks < sms * per_sm ? blocks : sms * per_sm);
    };
    auto per_sm = [](size_t all, size_t threads) { return static_cast<unsigned>(all / threads < 16 ? all / threads : 16); };
    if (cols <= 8192) {
        p.fused = true;
        const size_t threads = (cols + 7) / 8, ring = (cols + 15) / 16;
        p.group = static_cast<unsigned>(threads <= 32 ? 32 : (threads + 31) / 32 * 32);
        p.per_block = p.group == 32 ? 8 : 1;
        p.blocks = spread((rows + p.per_block - 1) / p.per_block, per_sm(1024, p.group * p.per_block));
        p.ring_group = static_cast<unsigned>((ring + 31) / 32 * 32);
        p.ring_per_sm = per_sm(512, p.ring_group);
        p.ring_blocks = spread(rows, p.ring_per_sm);
        p.workspace_floats = size_t(p.blocks > p.ring_blocks ? p.blocks : p.ring_blocks) * 3 * cols;
    } else {
        const size_t tiles = (cols + 255) / 256;
        size_t chunks = (sms * 8 + tiles - 1) / tiles;
        if (chunks > rows) chunks = rows;
        p.blocks = static_cast<unsigned>(chunks);
        p.workspace_floats = 2 * rows + chunks * 3 * cols;
    }
    return p;
}

namespace {

constexpr size_t kMaxRows = 0x7FFFFFFF;  // blocks of a grid

struct Array {
    const char *name;
    const void *p;
    size_t stride;
    bool output;
};

size_t size_of(rng_dtype t) { return t == RNG_F32 ? 4 : 2; }

rng_status check_types(const char *what, rng_dtype dtype, rng_dtype param)
{
    if (dtype != RNG_F32 && dtype != RNG_F16 && dtype != RNG_BF16)
        return fail(RNG_EINVAL, "%s: unknown dtype %d", what, dtype);
    if (param != dtype && param != RNG_F32)
        return fail(RNG_EINVAL, "%s: param_dtype %d is neither dtype nor RNG_F32", what, param);
    return RNG_OK;
}

rng_status check_vector(const char *what, const char *name, const void *p, size_t size)
{
    if (reinterpret_cast<uintptr_t>(p) % size != 0)
        return fail(RNG_EINVAL, "%s: %s is not aligned to its %zu-byte element", what, name, size);
    return RNG_OK;
}

// Whether two strided arrays share a byte.  With one stride, rows that lie
// side by side in it do not.
bool overlap(const Array &a, const Array &b, size_t rows, size_t cols, size_t size)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t a1 = a0 + ((rows - 1) * a.stride + cols) * size, b1 = b0 + ((rows - 1) * b.stride + cols) * size;
    if (a0 >= b1 || b0 >= a1) return false;
    if (a.stride == b.stride && rows > 1) {
        const size_t s = a.stride * size, d = (a0 > b0 ? a0 - b0 : b0 - a0) % s;
        if (d >= cols * size && s - d >= cols * size) return false;
    }
    return true;
}

// Addresses, strides and overlaps of the [rows, cols] arrays; in_place: the
// number of leading inputs that an output may be.
template <size_t N>
rng_status check_rows(const char *what, const Array (&a)[N], int in_place, size_t rows, size_t cols, size_t size)
{
    if (rows > kMaxRows) return fail(RNG_EINVAL, "%s: %zu rows exceed 2^31 - 1", what, rows);
    if (cols > 0x7FFFFFFF) return fail(RNG_EINVAL, "%s: %zu columns exceed 2^31 - 1", what, cols);
    for (const Array &x : a) {
        if (!x.p) continue;
        if (rng_status st = check_vector(what, x.name, x.p, size)) return st;
        if (rows > 1 && x.stride < cols)
            return fail(RNG_EINVAL, "%s: %s's stride %zu is below its %zu columns", what, x.name, x.stride, cols);
        const size_t room = (UINTPTR_MAX - reinterpret_cast<uintptr_t>(x.p)) / size;
        if (cols > room || (rows > 1 && x.stride > (room - cols) / (rows - 1)))
            return fail(RNG_EINVAL, "%s: %s runs past the end of the address space", what, x.name);
    }
    for (size_t i = 0; i < N; ++i) {
        if (!a[i].p || !a[i].output) continue;
        for (size_t j = 0; j < N; ++j) {
            if (j == i || !a[j].p || (a[j].output && j > i)) continue;
            const bool same = a[i].p == a[j].p && (a[i].stride == a[j].stride || rows == 1);
            if (static_cast<int>(j) < in_place && same) continue;
            if (overlap(a[i], a[j], rows, cols, size))
                return fail(RNG_EINVAL, "%s: %s and %s overlap", what, a[i].name, a[j].name);
        }
    }
    return RNG_OK;
}

// A contiguous array beside them: a weight, a row's statistic, the workspace.
struct Flat {
    const char *name;
    const void *p;
    size_t bytes;
    bool output;
};

// Whether a flat array shares a byte with a row: with the first one that ends
// past its beginning.
bool overlap(const Array &a, const Flat &f, size_t rows, size_t cols, size_t size)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), f0 = reinterpret_cast<uintptr_t>(f.p);
    const size_t used = cols * size, step = a.stride * size;
    const size_t row = f0 < a0 + used ? 0 : rows == 1 ? 1 : (f0 - a0 - used) / step + 1;
    return row < rows && a0 + row * step < f0 + f.bytes;
}

// Outputs share no byte with anything else (the [rows, cols] arrays among
// themselves are check_rows's).
template <size_t N, size_t M>
rng_status check_flat(const char *what, const Flat (&f)[M], const Array (&a)[N], size_t rows, size_t cols, size_t size)
{
    for (size_t i = 0; i < M; ++i) {
        if (!f[i].p || f[i].bytes == 0) continue;
        const uintptr_t at = reinterpret_cast<uintptr_t>(f[i].p);
        if (f[i].bytes > UINTPTR_MAX - at)
            return fail(RNG_EINVAL, "%s: %s runs past the end of the address space", what, f[i].name);
        for (const Array &x : a)
            if (rows && x.p && (x.output || f[i].output) && overlap(x, f[i], rows, cols, size))
                return fail(RNG_EINVAL, "%s: %s and %s overlap", what, x.name, f[i].name);
        for (size_t j = 0; j < i; ++j) {
            const uintptr_t other = reinterpret_cast<uintptr_t>(f[j].p);
            if (f[j].p && (f[i].output || f[j].output) && at < other + f[j].bytes && other < at + f[i].bytes)
                return fail(RNG_EINVAL, "%s: %s and %s overlap", what, f[j].name, f[i].name);
        }
    }
    return RNG_OK;
}

template <size_t N>
bool whole_vectors(const Array (&a)[N], size_t rows, size_t cols, size_t size)
{
    bool yes = cols * size % 16 == 0;
    for (const Array &x : a)
        if (x.p) yes = yes && reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && (rows == 1 || x.stride * size % 16 == 0);
    return yes;
}

bool on_vector(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

rng_status check_probability(const char *what, float p)
{
    if (!(p >= 0.0f && p < 1.0f)) return fail(RNG_EINVAL, "%s: p = %g is outside [0, 1)", what, (double)p);
    return RNG_OK;
}

// f(T, W) for the element types' tags.
template <class F>
cudaError_t with_types(rng_dtype dtype, rng_dtype param, F &&f)
{
    if (dtype == RNG_F32) return f(float{}, float{});
    if (dtype == RNG_F16) return param == RNG_F32 ? f(__half{}, float{}) : f(__half{}, __half{});
    return param == RNG_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}

}  // namespace
}  // namespace rngk

using namespace rngk;

extern "C" {

rng_status rng_dropout_layer_norm_fwd(const void *x, size_t x_stride, const void *bias, const void *residual,
                                      size_t residual_stride, const void *gamma, const void *beta, void *y,
                                      size_t y_stride, void *h, size_t h_stride, float *mean, float *rstd,
                                      size_t rows, size_t cols, rng_dtype dtype, rng_dtype param_dtype, float p,
                                      uint32_t seed, uint32_t first_counter, float eps, void *stream)
{
    static const char what[] = "rng_dropout_layer_norm_fwd";
    if (rng_status st = check_types(what, dtype, param_dtype)) return st;
    if (rng_status st = check_probability(what, p)) return st;
    if (!(eps >= 0.0f && std::isfinite(eps)))
        return fail(RNG_EINVAL, "%s: eps = %g is negative or not finite", what, (double)eps);
    if (rows == 0 || cols == 0) return RNG_OK;
    if (!x || !y) return fail(RNG_EINVAL, "%s: x or y is NULL", what);
    const size_t size = size_of(dtype), psize = size_of(param_dtype);
    const Array arrays[] = {{"x", x, x_stride, false},
                            {"residual", residual, residual_stride, false},
                            {"y", y, y_stride, true},
                            {"h", h, h_stride, true}};
    if (rng_status st = check_rows(what, arrays, 2, rows, cols, size)) return st;
    const void *weights[] = {bias, gamma, beta};
    for (const void *w : weights)
        if (rng_status st = check_vector(what, "a weight", w, psize)) return st;
    if (rng_status st = check_vector(what, "mean", mean, 4)) return st;
    if (rng_status st = check_vector(what, "rstd", rstd, 4)) return st;
    const Flat flat[] = {{"bias", bias, cols * psize, false},
                         {"gamma", gamma, cols * psize, false},
                         {"beta", beta, cols * psize, false},
                         {"mean", mean, rows * sizeof(float), true},
                         {"rstd", rstd, rows * sizeof(float), true}};
    if (rng_status st = check_flat(what, flat, arrays, rows, cols, size)) return st;
    clear_error();
    NormFwd a{};
    a.x = {x, x_stride}, a.residual = {residual, residual_stride}, a.y = {y, y_stride}, a.h = {h, h_stride};
    a.bias = bias, a.gamma = gamma, a.beta = beta, a.mean = mean, a.rstd = rstd;
    a.rows = rows, a.cols = static_cast<uint32_t>(cols), a.eps = eps, a.first = first_counter;
    a.mask = make_mask(p, seed);
    const bool vectors = whole_vectors(arrays, rows, cols, size) && on_vector(bias) && on_vector(gamma) && on_vector(beta);
    const cudaError_t e = with_types(dtype, param_dtype, [&](auto t, auto w) {
        return launch_norm_fwd<decltype(t), decltype(w)>(a, vectors, static_cast<cudaStream_t>(stream));
    });
    return e == cudaSuccess ? RNG_OK : cuda_fail(e, what);
}

size_t rng_dropout_layer_norm_bwd_workspace(size_t rows, size_t cols)
{
    return rows && cols ? norm_bwd_plan(rows, cols).workspace_floats * sizeof(float) : 0;
}

rng_status rng_dropout_layer_norm_bwd(const void *dy, size_t dy_stride, const void *h, size_t h_stride,
                                      const void *dh, size_t dh_stride, const void *gamma, const float *mean,
                                      const float *rstd, void *dx, size_t dx_stride, void *dresidual,
                                      size_t dresidual_stride, void *dgamma, void *dbeta, void *dbias, size_t rows,
                                      size_t cols, rng_dtype dtype, rng_dtype param_dtype, float p, uint32_t seed,
                                      uint32_t first_counter, void *workspace, size_t workspace_bytes, void *stream)
{
    static const char what[] = "rng_dropout_layer_norm_bwd";
    if (rng_status st = check_types(what, dtype, param_dtype)) return st;
    if (rng_status st = check_probability(what, p)) return st;
    if (cols == 0) return RNG_OK;
    const size_t size = size_of(dtype), psize = size_of(param_dtype);
    const void *weights[] = {gamma, dgamma, dbeta, dbias};
    for (const void *w : weights)
        if (rng_status st = check_vector(what, "a weight or its gradient", w, psize)) return st;
    const Array arrays[] = {{"dy", dy, dy_stride, false},        {"dh", dh, dh_stride, false},
                            {"h", h, h_stride, false},           {"dx", dx, dx_stride, true},
                            {"dresidual", dresidual, dresidual_stride, true}};
    if (rows) {
        if (!dy || !h || !mean || !rstd || !dx) return fail(RNG_EINVAL, "%s: dy, h, mean, rstd or dx is NULL", what);
        if (rng_status st = check_rows(what, arrays, 2, rows, cols, size)) return st;
        if (rng_status st = check_vector(what, "mean", mean, 4)) return st;
        if (rng_status st = check_vector(what, "rstd", rstd, 4)) return st;
        const size_t need = rng_dropout_layer_norm_bwd_workspace(rows, cols);
        if (!workspace || !on_vector(workspace) || workspace_bytes < need)
            return fail(RNG_EINVAL, "%s: workspace of %zu bytes at a 16-byte boundary wanted, %zu given", what, need,
                        workspace ? workspace_bytes : size_t(0));
    } else if (cols > 0x7FFFFFFF) {
        return fail(RNG_EINVAL, "%s: %zu columns exceed 2^31 - 1", what, cols);
    }
    const Flat flat[] = {{"gamma", gamma, cols * psize, false},
                         {"mean", mean, rows * sizeof(float), false},
                         {"rstd", rstd, rows * sizeof(float), false},
                         {"dgamma", dgamma, cols * psize, true},
                         {"dbeta", dbeta, cols * psize, true},
                         {"dbias", dbias, cols * psize, true},
                         {"workspace", workspace, rows ? rng_dropout_layer_norm_bwd_workspace(rows, cols) : 0, true}};
    if (rng_status st = check_flat(what, flat, arrays, rows, cols, size)) return st;
    clear_error();
    NormBwd a{};
    a.dy = {dy, dy_stride}, a.h = {h, h_stride}, a.dh = {dh, dh_stride};
    a.dx = {dx, dx_stride}, a.dresidual = {dresidual, dresidual_stride};
    a.gamma = gamma, a.mean = mean, a.rstd = rstd, a.dgamma = dgamma, a.dbeta = dbeta, a.dbias = dbias;
    a.rows = rows, a.cols = static_cast<uint32_t>(cols), a.first = first_counter, a.mask = make_mask(p, seed);
    a.workspace = static_cast<float *>(workspace);
    const bool vectors = rows && whole_vectors(arrays, rows, cols, size) && on_vector(gamma);
    const cudaError_t e = with_types(dtype, param_dtype, [&](auto t, auto w) {
        return launch_norm_bwd<decltype(t), decltype(w)>(a, vectors, static_cast<cudaStream_t>(stream));
    });
    return e == cudaSuccess ? RNG_OK : cuda_fail(e, what);
}

}  // extern "C"
