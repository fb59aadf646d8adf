// attention_bwd.cu -- attention backward (include/rng.h, rng_attention_bwd) on
// the tensor cores.
//
// Two kernels, each of which draws the probabilities and the mask again, so
// that every sum has one owner and no atomics: query_kernel (a block per 256
// queries, over the keys) gives dq, the bias table's gradient and each query's
// (lse, delta); key_kernel (a block per 128 keys, over the queries of all heads
// of the key head) gives dk and dv.  S and dP come from two products into TMEM
// by tiles of 128 x 64; the threads of one of two slots turn them into dS (and
// P), written back over S in 16 bits as the TMEM operand of the products
// that accumulate dq (dk, dv), while the tensor core works for the other slot.
// Two threads share a row, so that four warps a scheduler hide each other's
// latencies.
// The tile of 64 lets both slots' scores and both accumulators of a head
// dimension of 128 fit the 512 TMEM columns.
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace rngk {
namespace {

constexpr int kRows = 128, kCols = 64;  // a slot's tile
constexpr int kHalf = kCols / 2;        // columns of a thread
// 2 x 256 for the slots, then a TMA warp, an MMA warp, two that only fill the warpgroup
constexpr int kThreads = 640;
constexpr uint32_t kTmaWarp = 16, kMmaWarp = 17;
// registers: 640 threads start with 96 each; 4 x 104 + 64 = 5 x 96
constexpr int kSlotRegisters = 104, kOtherRegisters = 64;
constexpr uint32_t kRowsBox = 16384, kColsBox = 8192;  // bytes of 128 and of 64 rows of 64 elements
constexpr float kLog2e = 1.4426950408889634f;

// P's scale as the 16-bit operand of dv: f16 would lose the probabilities of
// long rows to its smallest step (2^-24), so they are held times 2^10; they are
// at most 1.
template <class T>
constexpr float kLift = 0.0f;
template <>
constexpr float kLift<__half> = 10.0f;

struct BwdParams {
    CUtensorMap q_rows, do_rows, k_cols, v_cols;  // query_kernel's
    CUtensorMap k_rows, v_rows, q_cols, do_cols;  // key_kernel's
    Attention a;
    int32_t pack, units, q_tiles, len_pad;
    // [batch heads][len_pad]: lse (in base two unless there is a bias; +inf for a query that sees nothing) and
    // delta; [heads][2 reach]: the bias by relative position; [batch heads][q_tiles][buckets]: sums of dS
    float2 *stats;
    float *bias, *sums;
};

// ---- dq ------------------------------------------------------------------------

template <int kDim, bool kSplitKeys>
struct QueryShape {
    static constexpr int kBoxes = kDim / 64;
    static constexpr int kTiles = kSplitKeys ? 1 : 2;
    static constexpr uint32_t kRowsBytes = kBoxes * kRowsBox, kColsBytes = kBoxes * kColsBox;
    static constexpr int kKeyStages = kDim == 64 ? 6 : kSplitKeys ? 5 : 3, kValueStages = kDim == 64 ? 4 : kSplitKeys ? 3 : 2;
    static constexpr uint32_t kDo = kTiles * kRowsBytes, kKeys = 2 * kDo, kValues = kKeys + kKeyStages * kColsBytes;
    static constexpr uint32_t kTable = kValues + kValueStages * kColsBytes;
};

// The relative positions of a bucket, lo .. hi (empty: lo > hi).
__device__ __forceinline__ void bucket_range(const Buckets &b, int32_t n, int32_t &lo, int32_t &hi)
{
    constexpr int32_t kFar = 1 << 30;
    const bool past = b.past && n >= b.past;
    const int32_t k = past ? n - b.past : n;
    const int32_t near = k == 0 ? 0 : b.starts[k - 1], far = k == b.count - 1 ? kFar : b.starts[k] - 1;
    if (n >= b.total) {
        lo = 1, hi = 0;
    } else if (past) {
        lo = max(near, 1), hi = far;
    } else {
        lo = -far, hi = -near;
        if (!b.past && k == 0) hi = kFar;  // one way: every key past the query
    }
}

template <class T, int kDim, bool kSplitKeys, bool kDrop, bool kBias>
__global__ void __launch_bounds__(kThreads, 1) query_kernel(const __grid_constant__ BwdParams p)
{
    using S = QueryShape<kDim, kSplitKeys>;
    extern __shared__ uint8_t dynamic[];
    __shared__ alignas(8) uint64_t bars[2 * (S::kKeyStages + S::kValueStages) + 8];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t stalled;
    __shared__ float diagonals[16][64];
    const Attention &a = p.a;
    const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
    uint8_t *smem = dynamic + ((1024u - (smem_address(dynamic) & 1023u)) & 1023u);
    const uint32_t base = smem_address(smem);
    float *table = reinterpret_cast<float *>(smem + S::kTable);

    // ---- the block's work
    int32_t unit, q_tile;
    if (a.causal) {  // the longest first
        unit = blockIdx.x % p.units, q_tile = p.q_tiles - 1 - blockIdx.x / p.units;
    } else {
        q_tile = blockIdx.x % p.q_tiles, unit = blockIdx.x / p.q_tiles;
    }
    const int32_t packs = a.heads / p.pack, b = unit / packs, pack = unit % packs;
    const int32_t head0 = pack * p.pack, head_kv = head0 / a.group;
    const int32_t rows_per = kRows / p.pack;
    const int32_t i0 = q_tile * S::kTiles * rows_per;
    const int32_t keys = keys_of(a, b), pos0 = first_position(a, keys);
    int32_t count[2];
    for (int s = 0; s < 2; ++s) {
        const int32_t last = min(i0 + (kSplitKeys ? 1 : s + 1) * rows_per, a.len_q) - 1;  // the slot's last query
        int32_t end = a.causal ? min(keys, pos0 + last + 1) : keys;
        if (!kSplitKeys && i0 + s * rows_per >= a.len_q) end = 0;
        count[s] = max(0, (end + kCols - 1) / kCols);
    }
    const int32_t tiles = max(count[0], count[1]);

    const uint32_t k_full = smem_address(bars), k_empty = k_full + 8 * S::kKeyStages, v_full = k_empty + 8 * S::kKeyStages,
                   v_empty = v_full + 8 * S::kValueStages, scored = v_empty + 8 * S::kValueStages, ready = scored + 16,
                   done = ready + 16, q_full = done + 8, tail = q_full + 8;
    if (threadIdx.x == 0) {
        stalled = 0;
        for (int s = 0; s < S::kKeyStages; ++s) barrier_init(k_full + 8 * s, 1), barrier_init(k_empty + 8 * s, 1);
        for (int s = 0; s < S::kValueStages; ++s) barrier_init(v_full + 8 * s, 1), barrier_init(v_empty + 8 * s, 1);
        for (int s = 0; s < 2; ++s) barrier_init(scored + 8 * s, 1), barrier_init(ready + 8 * s, 8);
        barrier_init(done, 1), barrier_init(q_full, 1), barrier_init(tail, 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc<512>(smem_address(&tmem_base));
    if (kBias) {  // the bias by relative position, head head0 (pack is 1)
        const int32_t reach = bias_reach(a.buckets);
        for (int32_t t = threadIdx.x; t < 2 * reach; t += kThreads) {
            table[t] = to_f32(static_cast<const T *>(a.table)[bucket_of(a.buckets, t - reach) * a.heads + head0]);
            if (b == 0 && q_tile == 0) p.bias[static_cast<int64_t>(head0) * 2 * reach + t] = table[t];
        }
    }
    if (q_tile == p.q_tiles - 1)  // what key_kernel reads past the last query
        for (int32_t t = threadIdx.x; t < p.pack * (p.len_pad - a.len_q); t += kThreads)
            p.stats[(static_cast<int64_t>(b) * a.heads + head0 + t % p.pack) * p.len_pad + a.len_q + t / p.pack] =
                make_float2(INFINITY, 0.0f);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base;
    if (warp >= kTmaWarp) {
        give_registers<kOtherRegisters>();
        if (warp == kTmaWarp) {
            // ---- TMA: q and do, then K_n and V_n
            const bool one = elect_one();
            if (one && tiles) {
                barrier_expect(q_full, 2 * S::kDo);
                for (int t = 0; t < S::kTiles; ++t)
                    for (int c = 0; c < S::kBoxes; ++c) {
                        const uint32_t o = t * S::kRowsBytes + c * kRowsBox;
                        tma_load_5d(base + o, &p.q_rows, q_full, c * 64, 0, i0 + t * rows_per, pack, b);
                        tma_load_5d(base + S::kDo + o, &p.do_rows, q_full, c * 64, 0, i0 + t * rows_per, pack, b);
                    }
            }
            for (int32_t n = 0; n < tiles; ++n) {
                const int32_t j0 = n * kCols;
                const uint32_t ks = n % S::kKeyStages, vs = n % S::kValueStages;
                if (!barrier_wait(k_empty + 8 * ks, (n / S::kKeyStages & 1u) ^ 1u, &stalled)) break;
                // keys past n(b) that the array holds: whatever they are, dS's zeros must meet zeros
                const bool past = j0 + kCols > keys && keys < a.len_k;
                const uint32_t on = past ? tail : k_full + 8 * ks, dst = base + S::kKeys + ks * S::kColsBytes;
                if (one) {
                    barrier_expect(on, S::kColsBytes);
                    for (int c = 0; c < S::kBoxes; ++c) tma_load_5d(dst + c * kColsBox, &p.k_cols, on, c * 64, 0, j0, head_kv, b);
                }
                if (past) {
                    if (!barrier_wait(tail, 0, &stalled)) barrier_drain(tail, 0);
                    uint8_t *rows = smem + S::kKeys + ks * S::kColsBytes;
                    for (int c = 0; c < S::kBoxes; ++c)
                        for (uint32_t o = max(0, keys - j0) * 128u + lane * 16u; o < kColsBox; o += 512u)
                            *reinterpret_cast<uint4 *>(rows + c * kColsBox + o) = make_uint4(0, 0, 0, 0);
                    fence_async_shared();
                    __syncwarp();
                    if (one) barrier_arrive(k_full + 8 * ks);
                }
                if (!barrier_wait(v_empty + 8 * vs, (n / S::kValueStages & 1u) ^ 1u, &stalled)) break;
                if (one) {
                    barrier_expect(v_full + 8 * vs, S::kColsBytes);
                    for (int c = 0; c < S::kBoxes; ++c)
                        tma_load_5d(base + S::kValues + vs * S::kColsBytes + c * kColsBox, &p.v_cols, v_full + 8 * vs, c * 64, 0,
                                    j0, head_kv, b);
                }
            }
            if (stalled && one)  // nothing may land after the block has ended
                for (int32_t n = max(0, tiles - S::kKeyStages); n < tiles; ++n)
                    for (uint32_t tries = 0;
                         tries < 100000 && !(barrier_try(k_full + 8 * (n % S::kKeyStages), n / S::kKeyStages & 1u) &&
                                             barrier_try(v_full + 8 * (n % S::kValueStages), n / S::kValueStages & 1u));
                         ++tries) {}
        } else if (warp == kMmaWarp) {
            // ---- MMA
            if (elect_one() && tiles) {
                constexpr uint32_t kScores = mma_shape<T>(kCols, false), kOut = mma_shape<T>(kDim, true);
                uint32_t given0 = 0, given1 = 0;
                auto scores = [&](int slot, int32_t n) {
                    const uint32_t ks = n % S::kKeyStages, vs = n % S::kValueStages;
                    const uint32_t q = base + (kSplitKeys ? 0 : slot) * S::kRowsBytes, k = base + S::kKeys + ks * S::kColsBytes,
                                   v = base + S::kValues + vs * S::kColsBytes;
                    barrier_wait_one(k_full + 8 * ks, n / S::kKeyStages & 1u, &stalled);
                    tmem_fence_after();
                    const uint64_t qd = row_major_tile(q), kd = row_major_tile(k), dd = row_major_tile(q + S::kDo), vd = row_major_tile(v);
#pragma unroll
                    for (int i = 0; i < kDim / 16; ++i)
                        mma_step(tmem + slot * 256, qd + row_step(i, kRowsBox), kd + row_step(i, kColsBox), kScores, i > 0);
                    barrier_wait_one(v_full + 8 * vs, n / S::kValueStages & 1u, &stalled);
                    tmem_fence_after();
#pragma unroll
                    for (int i = 0; i < kDim / 16; ++i)
                        mma_step(tmem + slot * 256 + kCols, dd + row_step(i, kRowsBox), vd + row_step(i, kColsBox), kScores, i > 0);
                    mma_commit(scored + 8 * slot);
                };
                auto product = [&](int slot, int32_t n, bool first) {
                    const uint32_t k = base + S::kKeys + n % S::kKeyStages * S::kColsBytes;
                    barrier_wait_one(ready + 8 * slot, (slot ? given1++ : given0++) & 1u, &stalled);
                    tmem_fence_after();
                    const uint64_t kd = column_major_tile(k, S::kBoxes > 1 ? kColsBox : 1024);
#pragma unroll
                    for (int i = 0; i < kCols / 16; ++i)
                        mma_step_tmem(tmem + slot * 256 + 2 * kCols, tmem + slot * 256 + i / 2 * kHalf + i % 2 * 8, kd + i * (2048 / 16), kOut,
                                      !first || i > 0);
                };
                auto release_k = [&](int32_t n) { mma_commit(k_empty + 8 * (n % S::kKeyStages)); };
                auto release_v = [&](int32_t n) { mma_commit(v_empty + 8 * (n % S::kValueStages)); };
                barrier_wait_one(q_full, 0, &stalled);
                if (kSplitKeys) {
#pragma unroll 1
                    for (int32_t n = -2; n < tiles; ++n) {
                        if (n >= 0) product(n & 1, n, n < 2), release_k(n);
                        if (n + 2 < tiles) scores(n & 1, n + 2), release_v(n + 2);
                    }
                } else {
#pragma unroll 1
                    for (int32_t n = -1; n < tiles; ++n) {
#pragma unroll 1
                        for (int s = 0; s < 2; ++s) {
                            if (n >= 0 && n < count[s]) product(s, n, n == 0);
                            if (n + 1 < count[s]) scores(s, n + 1);
                        }
                        if (n >= 0) release_k(n);
                        if (n + 1 < tiles) release_v(n + 1);
                    }
                }
                mma_commit(done);
            }
        }
    } else {
        take_registers<kSlotRegisters>();
        // ---- the slots' rows
        const int slot = warp / 8, half = warp / 4 % 2;
        const int32_t r = (warp % 4) * 32 + lane;
        const uint32_t lanes = (warp % 4) * 32u << 16;
        const uint32_t mine = tmem + slot * 256 + lanes + half * kHalf;  // the thread's scores, then its dS; dP kCols on
        const uint32_t out = tmem + slot * 256 + lanes + 2 * kCols + half * (kDim / 2);
        const int32_t row0 = kSplitKeys ? 0 : slot * kRows;
        const int32_t warp_i = i0 + (row0 + (warp % 4) * 32) / p.pack;
        const int32_t i = i0 + (row0 + r) / p.pack, head = head0 + r % p.pack;
        const bool valid = i < a.len_q, any = warp_i < a.len_q;
        const int32_t pos = pos0 + i;
        const int64_t index = (static_cast<int64_t>(b) * a.heads + head);
        const uint32_t counter = a.first + (static_cast<uint32_t>(index) * a.len_q + i) * static_cast<uint32_t>(a.len_k) + half * kHalf;
        const int32_t visible = a.causal ? min(keys, pos + 1) : keys;
        const int32_t warp_visible = a.causal ? min(keys, pos0 + warp_i + 1) : keys;
        const int32_t reach = bias_reach(a.buckets);
        const int32_t last_start = !kBias ? 0 : a.buckets.starts[a.buckets.count - 2];

        float lse = INFINITY, delta = 0.0f;
        if (valid) {
            const T *o = static_cast<const T *>(a.o) + b * a.os.batch + i * a.os.len + head * a.os.head;
            const T *d_o = static_cast<const T *>(a.d_o) + b * a.dos.batch + i * a.dos.len + head * a.dos.head;
            for (int32_t d = 0; d < a.dim; d += 8) {
                float x[8], y[8];
                unpack<T, 8>(load<false, T, 8>(o + d), x);
                unpack<T, 8>(load<false, T, 8>(d_o + d), y);
#pragma unroll
                for (int e = 0; e < 8; ++e) delta += x[e] * y[e];
            }
            lse = a.lse[index * a.len_q + i];
            // a query that sees nothing: exp(s - inf) = 0 whatever its scores
            lse = lse == -INFINITY ? INFINITY : kBias ? lse : lse * kLog2e;
            if (half == 0 && (slot == 0 || !kSplitKeys)) p.stats[index * p.len_pad + i] = make_float2(lse, delta);
        }

        float own[kMaxBuckets / 32] = {}, far_low = 0.0f, far_high = 0.0f;
        const float2 scale = make_float2(a.mask.scale, a.mask.scale), minus = make_float2(-delta, -delta);
        uint32_t turn = 0;
        for (int32_t n = kSplitKeys ? slot : 0; n < count[kSplitKeys ? 0 : slot]; n += kSplitKeys ? 2 : 1, ++turn) {
            const int32_t j0 = n * kCols + half * kHalf;
            barrier_wait(scored + 8 * slot, turn & 1u, &stalled);
            tmem_fence_after();
            if (any) {
                uint32_t v[2][32];  // S, then dP
                tmem_load32(v[0], mine);
                tmem_load32(v[1], mine + kCols);
                tmem_wait_load(v);
                uint32_t(&s)[32] = v[0], (&dp)[32] = v[1];
                const int32_t low = j0 - (pos0 + warp_i + 31), high = j0 + kHalf - 1 - (pos0 + warp_i);
                const bool far = high <= -last_start || low >= last_start;
                if (kBias) {
                    const float2 k2 = make_float2(a.scale, a.scale);
                    if (far) {
                        const float edge = table[high <= -last_start ? 0 : 2 * reach - 1];
#pragma unroll
                        for (int e = 0; e < kHalf; e += 2) {
                            const float2 f = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), k2, make_float2(edge, edge));
                            s[e] = __float_as_uint(f.x), s[e + 1] = __float_as_uint(f.y);
                        }
                    } else {
                        const float *t = table + (j0 - pos + reach);
#pragma unroll
                        for (int e = 0; e < kHalf; e += 2) {
                            const float2 f = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), k2, make_float2(t[e], t[e + 1]));
                            s[e] = __float_as_uint(f.x), s[e + 1] = __float_as_uint(f.y);
                        }
                    }
                }
                // P = exp(S - lse); dS = P (dP / (1 - p) - delta), dP dropped as P was
                const float2 to_base2 = kBias ? make_float2(kLog2e, kLog2e) : make_float2(a.scale * kLog2e, a.scale * kLog2e);
                const float2 l2 = make_float2(-lse, -lse);
                for_pairs32<kDrop>(a.mask, counter + n * kCols, [&](uint32_t e, float2 k) {
                    float2 f = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                    f = kBias ? mul2(add2(f, l2), to_base2) : fma2(f, to_base2, l2);
                    const float2 prob = make_float2(exp2_approx(f.x), exp2_approx(f.y));
                    float2 d = make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1]));
                    if (kDrop) d = mul2(d, k);
                    d = mul2(fma2(d, scale, minus), prob);
                    s[e] = __float_as_uint(d.x), s[e + 1] = __float_as_uint(d.y);
                });
                if (j0 + kHalf > warp_visible) {
                    const int32_t seen = visible - j0;
#pragma unroll
                    for (int e = 0; e < kHalf; ++e)
                        if (e >= seen) s[e] = 0;
                }
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pack2<T>(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
                tmem_store16(mine, w);
                tmem_wait_store();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(ready + 8 * slot);
                if (kBias && a.dtable) {
                    if (!valid) {
#pragma unroll
                        for (int e = 0; e < kHalf; ++e) s[e] = 0;
                    }
                    if (far) {  // one bucket
                        float2 total = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int e = 0; e < kHalf; e += 2) total = add2(total, make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])));
                        (high <= -last_start ? far_low : far_high) += total.x + total.y;
                    } else {
                        // sums along the diagonals of the warp's 32 x 32 tile: a partial sum moves one row down with
                        // each column; what leaves row 31, or is left in the last column, is a whole one
                        float acc = 0.0f;
#pragma unroll
                        for (int e = 0; e < kHalf; ++e) {
                            acc = __shfl_up_sync(0xFFFFFFFFu, acc, 1);
                            acc = (lane ? acc : 0.0f) + __uint_as_float(s[e]);
                            if (lane == 31) diagonals[warp][e] = acc;
                        }
                        if (lane < 31) diagonals[warp][62 - lane] = acc;
                        __syncwarp();
                        // diagonal d is relative position low + d; a lane adds the buckets lane, lane + 32, ...
#pragma unroll
                        for (int m = 0; m < kMaxBuckets / 32; ++m) {
                            if (32 * m < a.buckets.total) {
                                int32_t from, to;
                                bucket_range(a.buckets, lane + 32 * m, from, to);
                                from = max(from - low, 0), to = min(to - low, 62);
#pragma unroll 1
                                for (int32_t d = from; d <= to; ++d) own[m] += diagonals[warp][d];
                            }
                        }
                        __syncwarp();
                    }
                }
            } else if (lane == 0) {
                barrier_arrive(ready + 8 * slot);
            }
        }

        // ---- the result, through the tiles' memory, which nothing reads any more
        if (tiles) {
            barrier_wait(done, 0, &stalled);
            tmem_fence_after();
        }
        float *hand = reinterpret_cast<float *>(smem + S::kKeys);
        [[maybe_unused]] float *by_bucket = hand + kDim * kRows * (kSplitKeys ? 1 : 0);  // [16][kMaxBuckets]
        if (kBias && a.dtable) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) {
                far_low += __shfl_xor_sync(0xFFFFFFFFu, far_low, m);
                far_high += __shfl_xor_sync(0xFFFFFFFFu, far_high, m);
            }
#pragma unroll
            for (int m = 0; m < kMaxBuckets / 32; ++m) {
                const int32_t bucket = lane + 32 * m;
                if (bucket == a.buckets.count - 1) own[m] += far_low;
                if (bucket == (a.buckets.past ? a.buckets.total - 1 : 0)) own[m] += far_high;
                by_bucket[warp * kMaxBuckets + bucket] = own[m];
            }
        }
        const bool two = kSplitKeys && tiles > 1;
        if (two && slot == 1 && any) {
#pragma unroll 1
            for (int c = 0; c < kDim / 64; ++c) {
                uint32_t o[1][32];
                tmem_load32(o[0], out + 32 * c);
                tmem_wait_load(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) hand[(half * (kDim / 2) + 32 * c + e) * kRows + r] = __uint_as_float(o[0][e]);
            }
        }
        asm volatile("bar.sync 1, 512;" ::: "memory");
        if (kBias && a.dtable && threadIdx.x < a.buckets.total) {
            float s = 0.0f;
            for (int w = 0; w < 16; ++w) s += by_bucket[w * kMaxBuckets + threadIdx.x];
            p.sums[((static_cast<int64_t>(b) * a.heads + head0) * p.q_tiles + q_tile) * a.buckets.total + threadIdx.x] = s;
        }
        if (any && (!kSplitKeys || slot == 0)) {
            T *row = static_cast<T *>(a.dq) + b * a.dqs.batch + i * a.dqs.len + head * a.dqs.head;
            const bool has = count[kSplitKeys ? 0 : slot] > 0;
#pragma unroll 1
            for (int c = 0; c < kDim / 64; ++c) {
                uint32_t o[1][32] = {};
                const int col = half * (kDim / 2) + 32 * c;
                if (has) {
                    tmem_load32(o[0], out + 32 * c);
                    tmem_wait_load(o);
                }
                if (valid) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float eight[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            eight[k] = __uint_as_float(o[0][e + k]);
                            if (two) eight[k] += hand[(col + e + k) * kRows + r];
                            eight[k] *= a.scale;
                        }
                        if (col + e < a.dim) store<T, 8>(row + col + e, eight);
                    }
                }
            }
        }
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) tmem_free<512>(tmem);
}

// ---- dk, dv ----------------------------------------------------------------------

template <int kDim>
struct KeyShape {
    static constexpr int kBoxes = kDim / 64;
    static constexpr uint32_t kRowsBytes = kBoxes * kRowsBox, kColsBytes = kBoxes * kColsBox;
    static constexpr int kStages = kDim == 64 ? 8 : 4;
    static constexpr uint32_t kStageBytes = 2 * kColsBytes;          // q, do
    static constexpr uint32_t kRing = 2 * kRowsBytes;                // after k, v
    static constexpr uint32_t kStats = kRing + kStages * kStageBytes;  // kCols (lse, delta) a stage
    static constexpr uint32_t kBytes = kStats + kStages * kCols * sizeof(float2);
};

template <class T, int kDim, bool kDrop, bool kBias>
__global__ void __launch_bounds__(kThreads, 1) key_kernel(const __grid_constant__ BwdParams p)
{
    using S = KeyShape<kDim>;
    extern __shared__ uint8_t dynamic[];
    __shared__ alignas(8) uint64_t bars[2 * S::kStages + 6];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t stalled;
    const Attention &a = p.a;
    const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
    uint8_t *smem = dynamic + ((1024u - (smem_address(dynamic) & 1023u)) & 1023u);
    const uint32_t base = smem_address(smem);

    // ---- the block's work: the first keys, whose causal part is the longest, first
    const int32_t units = a.batch * a.heads_kv, unit = blockIdx.x % units;
    const int32_t b = unit / a.heads_kv, head_kv = unit % a.heads_kv;
    const int32_t j0 = blockIdx.x / units * kRows;
    const int32_t keys = keys_of(a, b), pos0 = first_position(a, keys);
    const int32_t q_tiles = (a.len_q + kCols - 1) / kCols;
    const int32_t first_i = a.causal && j0 > pos0 ? j0 - pos0 : 0;  // the first query that sees any of the keys
    const int32_t begin = min(first_i / kCols, q_tiles), per_head = j0 < keys ? q_tiles - begin : 0;
    const int32_t tiles = per_head * a.group;

    const uint32_t full = smem_address(bars), empty = full + 8 * S::kStages, scored = empty + 8 * S::kStages,
                   ready = scored + 16, done = ready + 16, k_full = done + 8;
    if (threadIdx.x == 0) {
        stalled = 0;
        for (int s = 0; s < S::kStages; ++s) barrier_init(full + 8 * s, 1), barrier_init(empty + 8 * s, 1);
        for (int s = 0; s < 2; ++s) barrier_init(scored + 8 * s, 1), barrier_init(ready + 8 * s, 8);
        barrier_init(done, 1), barrier_init(k_full, 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc<512>(smem_address(&tmem_base));
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base, dv_at = tmem + 4 * kCols, dk_at = dv_at + 128;
    if (warp >= kTmaWarp) {
        give_registers<kOtherRegisters>();
        if (warp == kTmaWarp) {
            // ---- TMA: k and v, then the queries' tiles, head by head
            if (elect_one() && tiles) {
                barrier_expect(k_full, 2 * S::kRowsBytes);
                for (int c = 0; c < S::kBoxes; ++c) {
                    tma_load_5d(base + c * kRowsBox, &p.k_rows, k_full, c * 64, 0, j0, head_kv, b);
                    tma_load_5d(base + S::kRowsBytes + c * kRowsBox, &p.v_rows, k_full, c * 64, 0, j0, head_kv, b);
                }
                for (int32_t n = 0; n < tiles; ++n) {
                    const uint32_t stage = n % S::kStages, bar = full + 8 * stage;
                    const int32_t head = head_kv * a.group + n / per_head, i0 = (begin + n % per_head) * kCols;
                    barrier_wait_one(empty + 8 * stage, (n / S::kStages & 1u) ^ 1u, &stalled);
                    barrier_expect(bar, S::kStageBytes + kCols * sizeof(float2));
                    const uint32_t dst = base + S::kRing + stage * S::kStageBytes;
                    for (int c = 0; c < S::kBoxes; ++c) {
                        tma_load_5d(dst + c * kColsBox, &p.q_cols, bar, c * 64, 0, i0, head, b);
                        tma_load_5d(dst + S::kColsBytes + c * kColsBox, &p.do_cols, bar, c * 64, 0, i0, head, b);
                    }
                    bulk_load(base + S::kStats + stage * kCols * sizeof(float2),
                              p.stats + (static_cast<int64_t>(b) * a.heads + head) * p.len_pad + i0, kCols * sizeof(float2), bar);
                }
                if (stalled)  // nothing may land after the block has ended
                    for (int32_t n = max(0, tiles - S::kStages); n < tiles; ++n)
                        for (uint32_t tries = 0; tries < 100000 && !barrier_try(full + 8 * (n % S::kStages), n / S::kStages & 1u); ++tries) {}
            }
        } else if (warp == kMmaWarp) {
            // ---- MMA
            if (elect_one() && tiles) {
                constexpr uint32_t kScores = mma_shape<T>(kCols, false), kOut = mma_shape<T>(kDim, true);
                barrier_wait_one(k_full, 0, &stalled);
#pragma unroll 1
                for (int32_t n = -2; n < tiles; ++n) {
                    const uint32_t slot = n & 1;
                    if (n >= 0) {  // dV += P^T dO, dK += dS^T Q
                        const uint32_t stage = n % S::kStages, q = base + S::kRing + stage * S::kStageBytes;
                        barrier_wait_one(ready + 8 * slot, n / 2 & 1u, &stalled);
                        tmem_fence_after();
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint64_t qd = column_major_tile(q + (x ? 0 : S::kColsBytes), S::kBoxes > 1 ? kColsBox : 1024);
#pragma unroll
                            for (int i = 0; i < kCols / 16; ++i)
                                mma_step_tmem(x ? dk_at : dv_at, tmem + slot * 2 * kCols + x * 16 + i / 2 * kHalf + i % 2 * 8,
                                              qd + i * (2048 / 16), kOut, n > 0 || i > 0);
                        }
                        mma_commit(empty + 8 * stage);
                    }
                    if (n + 2 < tiles) {  // S^T = K Q^T, dP^T = V dO^T
                        const uint32_t stage = (n + 2) % S::kStages, q = base + S::kRing + stage * S::kStageBytes;
                        barrier_wait_one(full + 8 * stage, (n + 2) / S::kStages & 1u, &stalled);
                        tmem_fence_after();
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint64_t kd = row_major_tile(base + x * S::kRowsBytes), qd = row_major_tile(q + x * S::kColsBytes);
#pragma unroll
                            for (int i = 0; i < kDim / 16; ++i)
                                mma_step(tmem + slot * 2 * kCols + x * kCols, kd + row_step(i, kRowsBox), qd + row_step(i, kColsBox), kScores,
                                         i > 0);
                        }
                        mma_commit(scored + 8 * slot);
                    }
                }
                mma_commit(done);
            }
        }
    } else {
        take_registers<kSlotRegisters>();
        // ---- the slots' rows: a key each
        const int slot = warp / 8, half = warp / 4 % 2;
        const int32_t j = j0 + (warp % 4) * 32 + lane, warp_j = j0 + (warp % 4) * 32;
        const uint32_t lanes = (warp % 4) * 32u << 16;
        const uint32_t mine = tmem + slot * 2 * kCols + lanes + half * kHalf;  // S^T, then P^T and dS^T; dP^T kCols on
        const bool any = warp_j < keys;
        const int32_t reach = bias_reach(a.buckets);
        const int32_t last_start = !kBias ? 0 : a.buckets.starts[a.buckets.count - 2];
        constexpr float kUnlift = kLift<T> != 0.0f ? 1.0f / 1024.0f : 1.0f;
        const float scale = a.mask.scale * kUnlift, to_base2 = a.scale * kLog2e;
        for (int32_t n = slot; n < tiles; n += 2) {
            const int32_t head = head_kv * a.group + n / per_head, i0 = (begin + n % per_head) * kCols + half * kHalf;
            const float4 *stats = reinterpret_cast<const float4 *>(smem + S::kStats + (n % S::kStages * kCols + half * kHalf) * sizeof(float2));
            barrier_wait(scored + 8 * slot, n / 2 & 1u, &stalled);
            tmem_fence_after();
            if (any) {
                uint32_t v[2][32];  // S^T, then dP^T
                tmem_load32(v[0], mine);
                tmem_load32(v[1], mine + kCols);
                tmem_wait_load(v);
                uint32_t(&s)[32] = v[0], (&dp)[32] = v[1];
                const int32_t rel = j - pos0 - i0;  // to the thread's first query
                const int32_t low = warp_j - pos0 - i0 - (kHalf - 1), high = warp_j + 31 - pos0 - i0;
                uint32_t c = a.first + ((static_cast<uint32_t>(b) * a.heads + head) * a.len_q + i0) * static_cast<uint32_t>(a.len_k) + j;
                if (kBias) {
                    const bool far = high <= -last_start || low >= last_start;
                    const float *bias = p.bias + static_cast<int64_t>(head) * 2 * reach;
                    const float2 k2 = make_float2(a.scale, a.scale);
                    if (far) {
                        const float edge = bias[high <= -last_start ? 0 : 2 * reach - 1];
#pragma unroll
                        for (int e = 0; e < kHalf; e += 2) {
                            const float2 f = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), k2, make_float2(edge, edge));
                            s[e] = __float_as_uint(f.x), s[e + 1] = __float_as_uint(f.y);
                        }
                    } else {
                        bias += rel + reach;
#pragma unroll
                        for (int e = 0; e < kHalf; e += 2) {
                            const float2 f = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), k2, make_float2(bias[-e], bias[-e - 1]));
                            s[e] = __float_as_uint(f.x), s[e + 1] = __float_as_uint(f.y);
                        }
                    }
                }
                if (a.causal && high > 0) {  // query i0 + e sees key j from e = rel on
#pragma unroll
                    for (int e = 0; e < kHalf; ++e)
                        if (e < rel) s[e] = __float_as_uint(-INFINITY);
                }
                // P = exp(S - lse), dropped for dv; dS = P (dropout(dP) - delta) for dk
#pragma unroll
                for (int e = 0; e < kHalf; e += 2) {
                    const float4 st = stats[e / 2];  // two queries' lse, delta
                    float2 f = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                    f = kBias ? fma2(add2(f, make_float2(-st.x, -st.z)), make_float2(kLog2e, kLog2e), make_float2(kLift<T>, kLift<T>))
                              : fma2(f, make_float2(to_base2, to_base2), make_float2(kLift<T> - st.x, kLift<T> - st.z));
                    const float2 prob = make_float2(exp2_approx(f.x), exp2_approx(f.y));
                    float2 kept2 = prob, d = make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1]));
                    if (kDrop) {
                        const float2 k = make_float2(kept(a.mask, c), kept(a.mask, c + static_cast<uint32_t>(a.len_k)));
                        c += 2 * static_cast<uint32_t>(a.len_k);
                        kept2 = mul2(kept2, k), d = mul2(d, k);
                    }
                    d = mul2(fma2(d, make_float2(scale, scale), make_float2(-st.y * kUnlift, -st.w * kUnlift)), prob);
                    s[e / 2] = pack2<T>(kept2.x, kept2.y);
                    dp[e / 2] = pack2<T>(d.x, d.y);
                }
                tmem_store16(mine, reinterpret_cast<const uint32_t(&)[16]>(v[0]));
                tmem_store16(mine + 16, reinterpret_cast<const uint32_t(&)[16]>(v[1]));
                tmem_wait_store();
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) barrier_arrive(ready + 8 * slot);
        }

        // ---- the result: slot 0's threads write dv, slot 1's dk
        if (tiles) {
            barrier_wait(done, 0, &stalled);
            tmem_fence_after();
        }
        if (warp_j < a.len_k) {
            const Strides &st = slot ? a.dks : a.dvs;
            T *row = static_cast<T *>(slot ? a.dk : a.dv) + b * st.batch + j * st.len + head_kv * st.head;
            const float weight = slot ? a.scale : scale;
#pragma unroll 1
            for (int c = 0; c < kDim / 64; ++c) {
                uint32_t o[1][32] = {};
                const int col = half * (kDim / 2) + 32 * c;
                if (tiles) {
                    tmem_load32(o[0], (slot ? dk_at : dv_at) + lanes + col);
                    tmem_wait_load(o);
                }
                if (j < a.len_k) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float eight[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) eight[k] = j < keys ? __uint_as_float(o[0][e + k]) * weight : 0.0f;
                        if (col + e < a.dim) store<T, 8>(row + col + e, eight);
                    }
                }
            }
        }
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) tmem_free<512>(tmem);
}

// ---- the table ---------------------------------------------------------------------

// dtable[n, head]: a block to each, its threads' sums over batch and query
// tiles added in a fixed order.
template <class T>
__global__ void __launch_bounds__(256) table_kernel(const __grid_constant__ BwdParams p)
{
    __shared__ float sums[8];
    const Attention &a = p.a;
    const int32_t n = blockIdx.x, head = blockIdx.y;
    float s = 0.0f;
    for (int64_t r = threadIdx.x; r < static_cast<int64_t>(a.batch) * p.q_tiles; r += 256)
        s += p.sums[((r / p.q_tiles * a.heads + head) * p.q_tiles + r % p.q_tiles) * a.buckets.total + n];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) s += sums[w];
        static_cast<T *>(a.dtable)[n * a.heads + head] = from_f32<T>(s);
    }
}

// ---- launching ------------------------------------------------------------------------

// How a call is cut, and where its workspace's parts begin (in floats).
struct BwdPlan {
    int32_t dim, pack, units, q_tiles, len_pad;
    bool split_keys;
    size_t bias, sums, floats;
};

BwdPlan bwd_plan(const Attention &a)
{
    BwdPlan f{};
    f.dim = a.dim <= 64 ? 64 : 128;
    f.pack = packed_heads(a);
    f.units = a.batch * (a.heads / f.pack);
    const int32_t rows_per = kRows / f.pack, tiles = (a.len_q + rows_per - 1) / rows_per;
    // one tile of queries to a block where two would leave SMs idle
    f.split_keys = tiles == 1 || static_cast<int64_t>(f.units) * ((tiles + 1) / 2) < sm_count();
    f.q_tiles = f.split_keys ? tiles : (tiles + 1) / 2;
    f.len_pad = (a.len_q + kCols - 1) / kCols * kCols;
    const size_t heads = static_cast<size_t>(a.batch) * a.heads;
    f.bias = 2 * heads * f.len_pad;
    f.sums = f.bias + (a.table ? static_cast<size_t>(a.heads) * 2 * bias_reach(a.buckets) : 0);
    f.floats = f.sums + (a.dtable ? heads * f.q_tiles * a.buckets.total : 0);
    return f;
}

template <class T, int kDim, bool kSplitKeys, bool kDrop, bool kBias>
cudaError_t launch_queries(const BwdParams &p, cudaStream_t s)
{
    const auto kernel = query_kernel<T, kDim, kSplitKeys, kDrop, kBias>;
    const size_t bytes = 1024 + QueryShape<kDim, kSplitKeys>::kTable + (kBias ? 2 * bias_reach(p.a.buckets) * sizeof(float) : 0);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(static_cast<int64_t>(p.units) * p.q_tiles), kThreads, bytes, s>>>(p);
    note_launch();
    return cudaGetLastError();
}

template <class T, int kDim, bool kDrop, bool kBias>
cudaError_t launch_keys(const BwdParams &p, cudaStream_t s)
{
    const auto kernel = key_kernel<T, kDim, kDrop, kBias>;
    const size_t bytes = 1024 + KeyShape<kDim>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
    const int64_t blocks = static_cast<int64_t>(p.a.batch) * p.a.heads_kv * ((p.a.len_k + kRows - 1) / kRows);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    kernel<<<static_cast<unsigned>(blocks), kThreads, bytes, s>>>(p);
    note_launch();
    return cudaGetLastError();
}

template <class T, int kDim, bool kDrop, bool kBias>
cudaError_t launch_both(const BwdParams &p, bool queries, bool keys, bool split_keys, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (queries) e = split_keys ? launch_queries<T, kDim, true, kDrop, kBias>(p, s) : launch_queries<T, kDim, false, kDrop, kBias>(p, s);
    if (e == cudaSuccess && keys) e = launch_keys<T, kDim, kDrop, kBias>(p, s);
    return e;
}

template <class T, int kDim>
cudaError_t launch_both(const BwdParams &p, bool queries, bool keys, bool split_keys, cudaStream_t s)
{
    const bool drop = p.a.mask.threshold != 0, bias = p.a.table != nullptr;
    if (drop)
        return bias ? launch_both<T, kDim, true, true>(p, queries, keys, split_keys, s)
                    : launch_both<T, kDim, true, false>(p, queries, keys, split_keys, s);
    return bias ? launch_both<T, kDim, false, true>(p, queries, keys, split_keys, s)
                : launch_both<T, kDim, false, false>(p, queries, keys, split_keys, s);
}

}  // namespace

cudaError_t stalled_waits_bwd(uint64_t *count)
{
    return cudaMemcpyFromSymbol(count, g_stalled_waits, sizeof(uint64_t));
}

size_t attention_bwd_workspace(const Attention &a) { return bwd_plan(a).floats * sizeof(float); }

template <class T>
cudaError_t launch_attention_bwd(const Attention &a, cudaStream_t s)
{
    const BwdPlan f = bwd_plan(a);
    BwdParams p{};
    p.a = a;
    p.pack = f.pack, p.units = f.units, p.q_tiles = f.q_tiles, p.len_pad = f.len_pad;
    float *ws = static_cast<float *>(a.workspace);
    p.stats = reinterpret_cast<float2 *>(ws), p.bias = ws + f.bias, p.sums = ws + f.sums;
    const bool has_q = a.batch && a.heads && a.len_q, has_k = a.batch && a.heads_kv && a.len_k;
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    cudaError_t e = cudaSuccess;
    auto map = [&](CUtensorMap *m, const void *x, const Strides &st, int32_t len, int32_t heads, int32_t pack, int32_t box) {
        if (e == cudaSuccess) e = make_heads_map(m, bf16, x, st, a.batch, len, heads, a.dim, pack, box);
    };
    if (has_q) {
        map(&p.q_rows, a.q, a.qs, a.len_q, a.heads, f.pack, kRows), map(&p.do_rows, a.d_o, a.dos, a.len_q, a.heads, f.pack, kRows);
        map(&p.q_cols, a.q, a.qs, a.len_q, a.heads, 1, kCols), map(&p.do_cols, a.d_o, a.dos, a.len_q, a.heads, 1, kCols);
    }
    if (has_k) {
        map(&p.k_rows, a.k, a.ks, a.len_k, a.heads_kv, 1, kRows), map(&p.v_rows, a.v, a.vs, a.len_k, a.heads_kv, 1, kRows);
        map(&p.k_cols, a.k, a.ks, a.len_k, a.heads_kv, 1, kCols), map(&p.v_cols, a.v, a.vs, a.len_k, a.heads_kv, 1, kCols);
    }
    if (static_cast<int64_t>(f.units) * f.q_tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (e == cudaSuccess)
        e = f.dim == 64 ? launch_both<T, 64>(p, has_q, has_k, f.split_keys, s) : launch_both<T, 128>(p, has_q, has_k, f.split_keys, s);
    if (e == cudaSuccess && a.dtable && a.heads) {
        table_kernel<T><<<dim3(a.buckets.total, a.heads), 256, 0, s>>>(p);
        note_launch();
        e = cudaGetLastError();
    }
    return e;
}

template cudaError_t launch_attention_bwd<__half>(const Attention &, cudaStream_t);
template cudaError_t launch_attention_bwd<__nv_bfloat16>(const Attention &, cudaStream_t);

}  // namespace rngk
