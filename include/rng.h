/*
 * rng.h -- C ABI of the GB300 (sm_103a) stateless counter-based random fills.
 *
 * Every output element is a pure function of (seed, counter): element i of a
 * fill takes the counter c_i = (first_counter + i) mod 2^32.  The generator is
 * the lowbias32 hash32 of the Phobos stdlib page "Random numbers" (section
 * hash32), in wrapping 32-bit arithmetic:
 *
 *   hash32(x)  = mix(mix(mix(x,16) * 0x7FEB352D, 15) * 0x846CA68B, 16),
 *                mix(x, s) = x ^ (x >> s) with a logical shift;
 *   D32(s, c)  = hash32(c ^ hash32(s))                  (section uniform);
 *   D64(s, c)  = D32(s, 2c) << 32 | D32(s, 2c + 1),      2c mod 2^32.
 *
 * Conventions shared by every call below.
 *   - Pointers are device pointers (cudaMalloc, torch CUDA tensors, managed
 *     memory) on the calling thread's current CUDA device.  The caller owns
 *     them; the library never allocates or frees an output.
 *   - Each output must be aligned to its element size.  No alignment beyond
 *     that is required: a start that is not 16-byte aligned is peeled off with
 *     scalar stores and the rest is written in whole 16-byte vectors.
 *   - `stream` is a cudaStream_t (NULL: the legacy default stream).  Calls are
 *     stream-ordered and asynchronous: they return once the work is enqueued.
 *   - n == 0 is a no-op that returns RNG_OK without touching any pointer.
 *     n may exceed 2^32; counters then wrap and values repeat with period
 *     2^32 (2^31 for the 64-bit and normal draws, which consume counters 2c
 *     and 2c + 1).
 *   - Errors.  RNG_EINVAL is returned before anything is enqueued: a NULL or
 *     misaligned pointer with n > 0, a pointer whose n elements would run
 *     past the end of the address space, a bound of 0, p outside [0, 1) or
 *     NaN, partially overlapping input and output.  RNG_ECUDA reports an error
 *     returned by the CUDA runtime while enqueuing (launch failure, invalid
 *     stream); faults of the device work itself surface at the caller's next
 *     synchronisation, as for any CUDA kernel.  RNG_ENOMEM reports a failed
 *     allocation of the library's own per-device ziggurat miss list.
 *     rng_last_error() gives a message for the calling thread's last error.
 *   - Every call is thread-safe, except that calls of
 *     rng_fill_normal_f64_noalloc whose work overlaps on the GPU race (see
 *     there).
 *   - The fills other than the two f64 normals keep no device state: their
 *     launches can be captured into a CUDA graph and replayed.
 *   - A fill cut at any element equals the whole fill: filling [a, b) with
 *     first_counter + a gives elements a..b-1 of the fill from first_counter.
 */
#ifndef LOWBIAS32_RNG_H
#define LOWBIAS32_RNG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int rng_status;
#define RNG_OK 0
#define RNG_EINVAL 1
#define RNG_ECUDA 2
#define RNG_ENOMEM 3

/* ---- uniform fills ------------------------------------------------------ */

/* out[i] = D32(seed, c_i).  Phobos "Random numbers", section uniform: the
 * hash of the counter keyed by the hashed seed. */
rng_status rng_fill_u32(uint32_t seed, uint32_t first_counter, size_t n, uint32_t *out,
                        void *stream);

/* out[i] = D64(seed, c_i): the draws at 2c_i (high word) and 2c_i + 1 (low
 * word), the counter pair randn consumes (Phobos "Random numbers", section
 * randn); tandem-cuda "Performance" row fill_u64 gives the fill. */
rng_status rng_fill_u64(uint32_t seed, uint32_t first_counter, size_t n, uint64_t *out,
                        void *stream);

/* out[i] = uniform(seed, c_i) = (D32 & 0x7FFFFF) * 2^-23, exactly: the low 23
 * bits on the 2^-23 grid in [0, 1) (Phobos "Random numbers", section uniform). */
rng_status rng_fill_f32(uint32_t seed, uint32_t first_counter, size_t n, float *out,
                        void *stream);

/* out[i] = (D64(seed, c_i) >> 11) * 2^-53, exactly: the top 53 bits on the
 * 2^-53 grid in [0, 1) (tandem-cuda "Performance", row fill_f64). */
rng_status rng_fill_f64(uint32_t seed, uint32_t first_counter, size_t n, double *out,
                        void *stream);

/* ---- narrow fills ----------------------------------------------------------- */
/* (tandem-cuda "Performance", rows fill_u16, fill_f16_bits, fill_u8 and
 * fill_bool, restated on hash32.)  Each element stays a pure function of its
 * counter; one 32-bit draw serves 4, 2 or 32 consecutive counters, the word
 * index wrapping with the counter. */

/* out[i] = byte (c_i & 3) of D32(seed, c_i >> 2), bits 8(c_i & 3) .. +7. */
rng_status rng_fill_u8(uint32_t seed, uint32_t first_counter, size_t n, uint8_t *out, void *stream);

/* out[i] = halfword (c_i & 1) of D32(seed, c_i >> 1), bits 16(c_i & 1) .. +15. */
rng_status rng_fill_u16(uint32_t seed, uint32_t first_counter, size_t n, uint16_t *out, void *stream);

/* out[i] = binary16 bits of m 2^-10, m the low 10 bits of the u16 element at
 * c_i: a uniform on the 2^-10 grid in [0, 1), exactly. */
rng_status rng_fill_f16(uint32_t seed, uint32_t first_counter, size_t n, uint16_t *out, void *stream);

/* out[i] = bit (c_i & 31) of D32(seed, c_i >> 5), one byte (0 or 1) per bit. */
rng_status rng_fill_bool(uint32_t seed, uint32_t first_counter, size_t n, uint8_t *out, void *stream);

/* ---- bounded integers: Lemire's multiply-shift with rejection ------------ */
/* (perturbation-kernel "Backends", section "Why the GPU can be exact";
 * tandem-cuda "Performance", bounded rows.)  For a w-bit word x the candidate
 * is floor(x * bound / 2^w); it is accepted when (x * bound) mod 2^w >=
 * 2^w mod bound (Lemire's exact threshold), which makes every value in
 * [0, bound) exactly equally likely.  A rejected element retries on its own
 * substream, keyed by its counter: the k-th retry word is hash32(k ^ K) with
 * K = hash32(c_i ^ hash32(hash32(seed) ^ P)), P = 0x42333220 ("B32 ") for
 * 32-bit and 0x42363420 ("B64 ") for 64-bit words, whose k-th word is
 * hash32(2k ^ K) << 32 | hash32((2k + 1) ^ K).  bound == 0 is RNG_EINVAL. */

/* out[i] = below32(bound) on the 32-bit draw D32(seed, c_i). */
rng_status rng_fill_u32_below(uint32_t seed, uint32_t first_counter, size_t n, uint32_t bound,
                              uint32_t *out, void *stream);

/* out[i] = below64(bound) on the 64-bit draw D64(seed, c_i). */
rng_status rng_fill_u64_below(uint32_t seed, uint32_t first_counter, size_t n, uint64_t bound,
                              uint64_t *out, void *stream);

/* out[i] = low + below32(bound), wrapped to int32 (two's complement)
 * (tandem-cuda "Performance", row "with a low bound into int32_t"). */
rng_status rng_fill_i32_range(uint32_t seed, uint32_t first_counter, size_t n, int32_t low,
                              uint32_t bound, int32_t *out, void *stream);

/* out[i] = low + below32(bound) into int64, wrapped (8-byte elements from
 * 32-bit draws; tandem-cuda "Performance", row "into int64_t"). */
rng_status rng_fill_i64_range32(uint32_t seed, uint32_t first_counter, size_t n, int64_t low,
                                uint32_t bound, int64_t *out, void *stream);

/* out[i] = low + below64(bound), wrapped to int64. */
rng_status rng_fill_i64_range(uint32_t seed, uint32_t first_counter, size_t n, int64_t low,
                              uint64_t bound, int64_t *out, void *stream);

/* ---- normals ------------------------------------------------------------- */

/* out[i] = randn(seed, c_i) = sqrt(-2 ln(1 - u0)) cos(2 pi u1) with u0 =
 * uniform(seed, 2c_i), u1 = uniform(seed, 2c_i + 1) (Phobos "Random
 * numbers", section randn): one value per counter, the cosine branch of
 * Box-Muller, |out| <= sqrt(46 ln 2) ~ 5.648.  Computed in f32: below u0 =
 * 2^-7 the series (1 + u0)^2 - 1 of -2 ln(1 - u0), above it the hardware
 * log2; the hardware square root; the hardware cosine on the angle 2 pi u1
 * in [0, 2 pi) (no half-turn shift as in tandem-sycl "Design", section
 * Normals: GB300's cosine is as accurate over the whole turn).  Each value is
 * within 4e-6 (1 + |z|) of the exact z. */
rng_status rng_fill_normal_f32(uint32_t seed, uint32_t first_counter, size_t n, float *out,
                               void *stream);

/* Paired Box-Muller: both branches of each uniform pair, one 64-bit draw
 * per two values (half the hashing of rng_fill_normal_f32).  With q = c_i >> 1,
 * u0 = uniform(seed, 2q), u1 = uniform(seed, 2q + 1), r = sqrt(-2 ln(1 - u0)):
 * out[i] = r cos(2 pi u1) for even c_i (= randn(seed, q)), r sin(2 pi u1) for
 * odd c_i.  The pages' randn keeps the cosine branch only (Phobos "Random
 * numbers", section randn); tandem-sycl "Design", section Normals, draws
 * Box-Muller pairs.  Same accuracy as rng_fill_normal_f32: within
 * 4e-6 (1 + |z|) of the exact value. */
rng_status rng_fill_normal_f32_pairs(uint32_t seed, uint32_t first_counter, size_t n, float *out,
                                     void *stream);

/* Precise f32 normal: randn's definition (u0 = uniform(seed, 2 c_i), u1 =
 * uniform(seed, 2 c_i + 1), z = sqrt(-2 ln(1 - u0)) cos(2 pi u1)) evaluated
 * in binary32 to a few ulp: the library's own -ln(1 - u0) (within 0.5035 ulp)
 * and cos(2 pi u1) (within 0.90 ulp), an IEEE square root, so out[i] is
 * within 2.5 ulp of the exact value and reproducible bit for bit.  An opt-in
 * variant with its own values: tandem-sycl "Design", section Normals, keeps a
 * precise f32 Box-Muller as a build option beside the default float normal.
 * rng_fill_normal_f32 is faster and within 4e-6 (1 + |z|). */
rng_status rng_fill_normal_f32_precise(uint32_t seed, uint32_t first_counter, size_t n, float *out,
                                       void *stream);

/* out[i] = standard normal from the 1024-layer Marsaglia-Tsang ziggurat on
 * the 64-bit draw D64(seed, c_i) (tandem-sycl "Design", section Normals).
 * Layer j = w & 1023, sign = bit 10, magnitude x = (w >> 11) 2^-53 X[j]
 * rounded once; x < X[j+1] is stored at once (99.57 % of elements).  The
 * rest (0.43 %) are appended to a device miss list and resolved by a second
 * kernel on the substream hash32(k ^ K), K = hash32(c_i ^ hash32(hash32(seed)
 * ^ 0x4E363420)) ("N64 "): the base layer samples the tail beyond r =
 * X[1] (Marsaglia 1964), the others take the wedge test against exp(-x^2/2)
 * and otherwise start over with a fresh 64-bit word.  Both exp and log of
 * that path are fixed IEEE operation sequences, so the result is bit-exact
 * and reproducible.  The layer tables are static device data of the library
 * (no allocation).  The miss list (4 bytes per expected miss plus slack) is
 * the one device allocation: made per device on first use, grown when a
 * longer fill needs more, and held until the process exits; fills on
 * different streams that share it are ordered through its last event.  If
 * the list overflows, the second kernel walks the whole fill again. */
rng_status rng_fill_normal_f64(uint32_t seed, uint32_t first_counter, size_t n, double *out,
                               void *stream);

/* Allocation-free variant of rng_fill_normal_f64, for callers that cannot
 * call cudaMalloc: code whose device memory is entirely owned by another
 * allocator (a framework's caching allocator that reserved the pool up front,
 * where a cudaMalloc of ours would fail or fragment it), and latency-critical
 * paths that cannot accept cudaMalloc's implicit device synchronisation.  The
 * pages have no counterpart: it exists for those callers only.
 *   - Same values as rng_fill_normal_f64, bit for bit.
 *   - The miss counter and list live in one static device array of the
 *     library (8 MiB + 256 bytes, present on every device that loads the
 *     library until the process exits); the call makes no device allocation.
 *   - n must not exceed 2^28 elements; larger n returns RNG_EINVAL.
 *   - The first call on a device looks up the array's device address (with
 *     that device current); make that first call before any stream capture.
 *     The address is kept for the rest of the process: it assumes that the
 *     device's primary context is not reset (cudaDeviceReset) meanwhile.
 *   - Every call shares the array and clears its counter first: calls whose
 *     work overlaps on the GPU (other streams, other threads) race on it and
 *     give unspecified values.  Order them on one stream or with events.
 *   - Otherwise as rng_fill_normal_f64 (device pointers, stream-ordered). */
rng_status rng_fill_normal_f64_noalloc(uint32_t seed, uint32_t first_counter, size_t n, double *out,
                                       void *stream);

/* ---- exponentials (tandem-sycl "Design", section Exponentials) ------------ */

/* out[i] = -ln(1 - u), u = uniform(seed, c_i): 1 - u = V 2^-23 exact in
 * (0, 1], and the library's own table-driven binary32 logarithm of it
 * (neg_log_grid in include/rng_device.cuh: exact reduction by 8-bit
 * reciprocals, a TwoSum and a series to r^5, one final rounding), within
 * 0.5035 ulp of the exact value on every input and reproducible bit for bit;
 * in [0, 23 ln 2]. */
rng_status rng_fill_exponential_f32(uint32_t seed, uint32_t first_counter, size_t n, float *out,
                                    void *stream);

/* out[i] = -ln(1 - u), u = (D64(seed, c_i) >> 11) 2^-53, by neglog64: a
 * fixed-point logarithm in 32-, 64- and 128-bit integer arithmetic with no
 * FP64 arithmetic (one u64 -> f64 conversion rounds the result).  1 - u =
 * V 2^-53 with the integer V = 2^53 - m is reduced exactly by 2048 one-sided
 * reciprocals (r in [0, 1.5 2^-11)), log1p of the reduced argument is a
 * Horner series to r^5 in fixed point, the exponent and table terms are added
 * at scale 2^96, and the sum is rounded once to binary64; below u = 2^-12 the
 * value is the series in u itself.  Within 0.5007 ulp of -ln(1 - u),
 * reproducible bit for bit, in [0, 53 ln 2]; +0 at u = 0.  Bound by the
 * integer pipes on GB300. */
rng_status rng_fill_exponential_f64(uint32_t seed, uint32_t first_counter, size_t n, double *out,
                                    void *stream);

/* ---- dropout (Phobos "Random numbers", section dropout) ------------------- */

/* y[i] = uniform(seed, c_i) >= p ? x[i] / (1 - p) : +0, in f32 with IEEE
 * division; 1 - p is rounded to f32 first; a tie u == p is kept.  p must lie
 * in [0, 1).  x and y may be the same array (in place) but must not overlap
 * otherwise.  Reads 4 and writes 4 bytes per element. */
rng_status rng_dropout_fwd(const float *x, float *y, float p, uint32_t seed,
                           uint32_t first_counter, size_t n, void *stream);

/* dx[i] = the same mask applied to dy[i], redrawn from the same seed and
 * counters instead of stored (the page's backward pass): bit-for-bit the
 * forward computation on dy. */
rng_status rng_dropout_bwd(const float *dy, float *dx, float p, uint32_t seed,
                           uint32_t first_counter, size_t n, void *stream);

/* ---- a transformer layer's dropout, fused with what surrounds it ----------- */
/* The mask is dropout's above and is stored in neither direction: element e of
 * a masked array, e its flat index, is kept iff uniform(seed, first_counter +
 * e) >= p, and a kept value is multiplied by the binary32 value of 1 / (1 - p)
 * (rng_dropout_fwd divides by 1 - p: the last bit may differ).  p = 0 draws
 * nothing.  Sums and statistics are binary32, and an output is rounded once to
 * its type; attention also rounds the operands of its products, as said there. */

/* Element types. */
typedef int rng_dtype;
#define RNG_F32 0
#define RNG_F16 1
#define RNG_BF16 2

/* Bias, dropout, residual and layer norm of a [rows, cols] array:
 *
 *   h = residual + dropout(x + bias)           e = row * cols + column
 *   mean, rstd = mean of h's row, 1 / sqrt(variance + eps)
 *   y = (h - mean) * rstd * gamma + beta
 *
 * x, residual, y and h have type `dtype`; bias, gamma and beta (cols each)
 * have type `param_dtype`, which is dtype or RNG_F32; mean and rstd (rows
 * each) are f32.  bias, residual, gamma, beta, h, mean and rstd may be NULL
 * (0, 0, 1, 0, not stored, not stored, not stored).  The norm is taken of the
 * unrounded h.  Rows start x_stride, ... elements apart (a stride is not
 * looked at for a NULL array); columns are adjacent.
 * y and h may each be x's or residual's own array (same address and stride);
 * any other overlap of an output (mean and rstd among them) with another array
 * is RNG_EINVAL, as are a stride below cols (with rows > 1), a missing x or y, p
 * outside [0, 1) and a negative or non-finite eps.  rows == 0 or cols == 0 is a
 * no-op. */
rng_status rng_dropout_layer_norm_fwd(const void *x, size_t x_stride, const void *bias, const void *residual,
                                      size_t residual_stride, const void *gamma, const void *beta, void *y,
                                      size_t y_stride, void *h, size_t h_stride, float *mean, float *rstd,
                                      size_t rows, size_t cols, rng_dtype dtype, rng_dtype param_dtype, float p,
                                      uint32_t seed, uint32_t first_counter, float eps, void *stream);

/* Its gradient.  From dy, the stored h, mean and rstd, and dh (NULL: 0), the
 * gradient that reaches h past the norm:
 *
 *   g  = dy * gamma,  n = (h - mean) * rstd
 *   dz = rstd * (g - mean(g) - n * mean(g * n)) + dh
 *   dresidual = dz,   dx = dropout(dz)  (the forward mask, redrawn)
 *   dgamma = sum over rows of dy * n,  dbeta = of dy,  dbias = of dx
 *
 * dresidual, dgamma, dbeta and dbias may be NULL (not wanted); dgamma, dbeta
 * and dbias have type param_dtype, are summed in f32 in an order that depends
 * on the sizes and alignment alone, and are written (not added to): zeros for rows == 0.
 * dx and dresidual may each be dy's or dh's own array.  `workspace` holds
 * rng_dropout_layer_norm_bwd_workspace(rows, cols) bytes at a 16-byte
 * boundary (NULL where that is 0); it belongs to the call until its work is
 * done.  Other errors as above; a workspace that is too small is RNG_EINVAL. */
rng_status rng_dropout_layer_norm_bwd(const void *dy, size_t dy_stride, const void *h, size_t h_stride,
                                      const void *dh, size_t dh_stride, const void *gamma, const float *mean,
                                      const float *rstd, void *dx, size_t dx_stride, void *dresidual,
                                      size_t dresidual_stride, void *dgamma, void *dbeta, void *dbias, size_t rows,
                                      size_t cols, rng_dtype dtype, rng_dtype param_dtype, float p, uint32_t seed,
                                      uint32_t first_counter, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace that rng_dropout_layer_norm_bwd needs on the current device. */
size_t rng_dropout_layer_norm_bwd_workspace(size_t rows, size_t cols);

/* Attention with a learned relative position bias by buckets and dropout on
 * its probabilities.  For batch b, query i, head a (of heads_q; it reads key
 * head a / (heads_q / heads_kv)) and key j:
 *
 *   s = scale * <q, k> + bias_table[rng_relative_bucket(j - pos(i)), a]
 *   P = softmax over the visible j of s,  lse = log of the sum of exp(s)
 *   o = sum over j of dropout(P) v,       e = ((b heads_q + a) len_q + i) len_k + j
 *
 * pos(i) = i, or with queries_last i + n(b) - len_q (the queries are the last
 * len_q of the keys: a decoding step, a later piece of a prompt).  Key j is
 * visible iff j < n(b) and, when causal, j <= pos(i).  n(b) is
 * key_lengths[b], taken into [0, len_k], or len_k without key_lengths.  Keys
 * at or past n(b) have no influence, whatever their bits.  A query that sees
 * no key gets o = 0, lse = -inf and passes no gradient, whatever q and d_o hold
 * there.
 *
 * The struct holds device pointers and sizes; it is read during the call
 * only.  q, k, v, o (and their gradients) are [batch, length, heads,
 * head_dim] arrays of type dtype (RNG_F16 or RNG_BF16) whose strides are
 * given in elements in the order batch, length, head; head_dim is adjacent.
 * Each address is a multiple of 16 bytes and each stride of 8 elements (of a
 * dimension of size 1, any); head_dim is a multiple of 8 up to 128; heads_q
 * is a multiple of heads_kv.  bias_table (NULL: none) is [num_buckets,
 * heads_q] of type dtype, contiguous.  lse is [batch, heads_q, len_q] f32.
 *
 * s, the softmax statistics and all sums are f32; P (before its division by
 * the row's sum) and, in the backward pass, P and dS are rounded to dtype as
 * the operands of the matrix products that follow; where len_q * len_k *
 * heads_q is at most 65536, as two terms each, the value and what its rounding
 * left (whatever the batch).  The forward pass may split a long key axis by the
 * number of batch entries, which changes the order of its f32 sums.  In f16, dS
 * has f16's range: it is in steps of 2^-24 below 2^-14 and infinite above 65504,
 * so gradients that small or large want their loss scaled, as f16 outputs do.
 *
 * Any other NaN or infinity in q, k, v or d_o reaches what sees it; where a
 * causal mask ends inside a tile (128 queries or keys by 64) it may also reach
 * what is beside it there: the mask gives a weight of 0, and 0 times it is NaN. */
typedef struct rng_attention_args {
    rng_dtype dtype;
    int32_t batch, len_q, len_k, heads_q, heads_kv, head_dim;
    const void *q, *k, *v;
    int64_t q_stride[3], k_stride[3], v_stride[3];
    void *o; /* backward: read */
    int64_t o_stride[3];
    float *lse; /* forward: may be NULL; backward: read */
    const int32_t *key_lengths; /* [batch] or NULL */
    int32_t causal, queries_last;
    float scale;
    const void *bias_table; /* or NULL */
    int32_t num_buckets, max_distance, bidirectional;
    float p;
    uint32_t seed, first_counter;
    /* backward only */
    const void *d_o;
    void *dq, *dk, *dv;
    int64_t do_stride[3], dq_stride[3], dk_stride[3], dv_stride[3];
    void *dbias_table; /* [num_buckets, heads_q] of type dtype, written; or NULL */
    /* both: rng_attention_{fwd,bwd}_workspace(args) bytes at a 16-byte boundary */
    void *workspace;
    size_t workspace_bytes;
} rng_attention_args;

/* Forward: o and lse.  RNG_EINVAL: what the struct's description rules out, p
 * outside [0, 1), a scale that is not finite, num_buckets and max_distance
 * that rng_relative_bucket refuses (with a table), a length or batch * heads_q
 * above 2^30, an output (or the workspace) that overlaps any other array.  An
 * empty output is a no-op; len_k == 0 with queries gives o = 0. */
rng_status rng_attention_fwd(const rng_attention_args *args, void *stream);

/* Backward: dq, dk, dv and dbias_table from d_o and the forward's o and lse;
 * with delta = <d_o, o> and dP = dropout of <d_o, v>,
 *   dS = P (dP - delta),  dq = scale sum_j dS k,  dk = scale sum_i dS q,
 *   dv = sum_i dropout(P) d_o,  dbias_table[n, a] = sum of dS in bucket n.
 * dk and dv of a key head are summed over its query heads.  No atomics: the
 * results are the same bits every time.  P = exp(s - lse); where biases leave
 * nothing of the sum in an f32 lse (above 2^17, which bf16 has), the sum is
 * taken again, so that a row's P add up to 1 there too (slowly: one thread a
 * query). */
rng_status rng_attention_bwd(const rng_attention_args *args, void *stream);

/* Bytes of workspace on the current device (sizes, scale and
 * whether bias_table and dbias_table are NULL are looked at). */
size_t rng_attention_fwd_workspace(const rng_attention_args *args);
size_t rng_attention_bwd_workspace(const rng_attention_args *args);

/* The bucket of a relative position (key's minus query's).  With one
 * direction's count m = num_buckets / 2 when bidirectional, else num_buckets:
 * distance d < m / 2 has its own bucket d; above, bucket m / 2 + floor((m -
 * m / 2) ln(d / (m / 2)) / ln(max_distance / (m / 2))), at most m - 1, by
 * whole-number arithmetic.  Bidirectional: keys past the query use buckets m
 * and up; otherwise their distance is 0.  RNG_EINVAL: num_buckets outside
 * 2 (4 when bidirectional) .. 128 or odd when bidirectional, max_distance
 * outside m / 2 + 1 .. 1024, bucket == NULL. */
rng_status rng_relative_bucket(int64_t relative_position, int32_t num_buckets, int32_t max_distance,
                               int32_t bidirectional, int32_t *bucket);

/* ---- status -------------------------------------------------------------- */

/* A static string naming the status code. */
const char *rng_status_string(rng_status status);

/* The calling thread's message for its last non-OK status (static storage
 * per thread; "" when none). */
const char *rng_last_error(void);

/* ---- test and measurement hooks ------------------------------------------ */

/* Caps the number of entries the ziggurat miss list may hold (0 forces every
 * normal_f64 fill through the whole-fill walk of the second kernel);
 * SIZE_MAX restores the default capacity.  Applies to later fills on every
 * device. */
rng_status rng_debug_set_miss_capacity(size_t capacity);

/* Number of entries the most recent normal_f64 fill's table pass listed on
 * the current device (of its last chunk of at most 2^31 elements; above the
 * capacity when the list overflowed): every draw that misses the fast path,
 * plus the few fast draws the table pass leaves to the second kernel (those
 * its integer product cannot round, about 1e-4 of the elements, and about
 * 1e-6 whose product shares X[j+1]'s high word).  Synchronises the device. */
rng_status rng_debug_last_miss_count(uint64_t *count);

/* Number of kernels this library has launched since it was loaded, over all
 * devices and threads. */
uint64_t rng_debug_launch_count(void);

/* Evaluates the library's own binary64 functions on the device, out[i] =
 * f(in[i]) for i < n (in and out device arrays of doubles): the normal_f64
 * slow path's exp (which = 0) or log (which = 1), or (which = 2) the f64
 * exponential's fixed-point -ln(1 - m 2^-53) with m the low 53 bits of
 * in[i]'s bit pattern.  which = 3 and 4 take in[i]'s bit pattern as a 64-bit
 * ziggurat draw w and return its fast-path magnitude RNE((w >> 11) 2^-53
 * X[w & 1023]): by the table pass's integer product (NaN for a draw it
 * defers to the miss pass) and by its fma.  For checking those functions on
 * chosen inputs; which outside 0 .. 4 is RNG_EINVAL. */
rng_status rng_debug_eval_f64(int which, const double *in, double *out, size_t n, void *stream);

/* Number of waits inside the layer kernels (attention, layer norm) that ran out on the current
 * device since the library was loaded.  Every wait of theirs (for a tile, for
 * a product) ends after about two seconds at most, so that a fault of theirs
 * never holds the GPU; a count above 0 says that outputs are not to be
 * trusted.  Synchronises the device. */
rng_status rng_debug_stalled_waits(uint64_t *count);

/* A measurement aid with no counterpart on the pages: the write ceiling the
 * fills are compared with.  which = 0 enqueues cudaMemsetAsync(buf, 0x5A,
 * bytes); which = 1 launches the plainest 16-byte store kernel over buf, in
 * the launch shape of the fills (buf 16-byte aligned, bytes a multiple of
 * 16).  buf is a caller-owned device buffer whose contents are overwritten;
 * stream-ordered on stream.  RNG_EINVAL for another which, buf == NULL with
 * bytes > 0, buf + bytes past the end of the address space, or (which = 1) a
 * misaligned buf or size; bytes == 0 is a no-op. */
rng_status rng_debug_write_ceiling(int which, void *buf, size_t bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIAS32_RNG_H */
