// attention_bwd.cu -- attention backward (include/rng.h, rng_attention_bwd) on
// the tensor cores.
//
// Two kernels, each of which draws the probabilities and the mask again, so
// that every sum has one owner and no atomics: query_kernel (an item of work per
// 128 queries, over the keys) gives dq, the bias table's gradient and each
// query's (lse, delta); key_kernel (an item per 128 keys, over the queries of all
// heads of the key head) gives dk and dv.  S and dP come from two products into
// TMEM by tiles of 128 x 64; threads turn them into dS (and P), written back
// over S (and dP) in 16 bits as the TMEM operands of the products that accumulate
// dq (dk, dv).
//
// Such a tile is a chain of product, exponential and mask, product; several are
// under way at once, so that the tensor core works for some while others compute.
// TMEM's 512 columns hold the accumulators and three tiles' S and dP (two in
// key_kernel with a head dimension of 128).  A warpgroup takes a chain's tiles, a
// thread to a row; where there are two chains only, two warpgroups share a tile,
// 32 columns a thread, for as many warps.  A block that has finished takes over
// the work of one that has not started.
//
// What bounds them, measured (bf16, p = 0.1): both draw the mask, so instruction
// issue, 18 to 23 instructions a pair each.
//   16 x 1024 positions, 16 heads of 64, 32 buckets: query_kernel 254 us (issue slots
//     61 % busy, ALU pipe 41 %, tensor core 18 %), key_kernel 250 us (67, 47, 24 %),
//     table_kernel 5 us.
//   2 x 4096 causal positions, 16 heads of 128 over 4 key heads: query_kernel 238 us
//     (55, 39, 37 %), key_kernel 264 us (68, 47, 51 %).
//   24 x 77 x 115 ragged, 6 heads of 40, 20 buckets, f16: 12, 12 and 4 us, one after
//     the other and each mostly its own set-up.
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace rngk {
namespace {

constexpr int kRows = 128, kCols = 64;  // a tile

// The warpgroups of a block, and their registers: it starts with 65536 / threads
// a thread, the last warpgroup (a TMA warp, an MMA warp,
// two that only fill it) gives some to the others.
template <int kChains, int kShare>  // warpgroups of a tile
struct Crew {
    static constexpr int kGroups = kChains * kShare, kWorkers = 128 * kGroups, kThreads = kWorkers + 128;
    static constexpr uint32_t kTmaWarp = 4 * kGroups, kMmaWarp = kTmaWarp + 1;
    // 512 threads start with 128 each, 3 x 152 + 56 = 4 x 128; 640 with 96, 4 x 104 + 64 = 5 x 96
    static constexpr int kWorkerRegisters = kGroups == 3 ? 152 : 104, kOtherRegisters = kGroups == 3 ? 56 : 64;
    static_assert(kGroups == 3 || kGroups == 4, "");
};

constexpr uint32_t kRowsBox = 16384, kColsBox = 8192;  // bytes of 128 and of 64 rows of 64 elements
constexpr float kLog2e = 1.4426950408889634f;

// P's scale as the 16-bit operand of dv: f16 would lose the probabilities of
// long rows to its smallest step (2^-24), so they are held times 2^10; they are
// at most 1.
template <class T>
constexpr float kLift = 0.0f;
template <>
constexpr float kLift<__half> = 10.0f;
template <class T>
constexpr float kUnlift = kLift<T> != 0.0f ? 1.0f / 1024.0f : 1.0f;

struct BwdParams {
    CUtensorMap q_rows, do_rows, k_cols, v_cols;  // query_kernel's
    CUtensorMap k_rows, v_rows, q_cols, do_cols;  // key_kernel's
    Attention a;
    int32_t pack, pack_log, units, q_tiles, len_pad;
    Divider by_units, by_q_tiles, by_packs, by_group, by_key_units, by_heads_kv;
    // [batch heads][len_pad]: what key_kernel adds to a query's scores in base two, kLift - lse (with a bias, -lse
    // in the natural base; -inf for a query that sees nothing), and to its scaled dP, -delta; [heads][2 reach]: the bias by relative position; [batch heads][q_tiles][buckets]: sums of dS
    float2 *stats;
    float *bias, *sums;
    uint8_t *lost;  // [batch heads][len_pad / 32]: whether 32 queries have one whose lse is too large (below)
};

// Above 2^17 an f32 lse is 2^-7 and more off.  With a bias of the type's lowest
// value (or highest, or the 1e9 of additive masks) for all that a query sees,
// nothing is left in it of the logarithm of the sum of exp(s - largest s), and
// P = exp(s - lse) would be too large by the number of such keys.  Only bf16 has
// such values.  The sum of such a row's P is then taken again from its scores,
// and divides them: in query_kernel with the factors of dP and delta, in
// key_kernel by the row's first statistic, -log of the sum, after lse has been
// taken from the scores of a tile that has such rows.  Seldom, so as simply as
// can be; a byte for 32 queries is all that it costs others.
template <class T, bool kBias>
constexpr bool kMayLose = kBias && std::is_same<T, __nv_bfloat16>::value;
constexpr float kLostFrom = 131072.0f;
__device__ __forceinline__ bool loses(float lse) { return fabsf(lse) >= kLostFrom && fabsf(lse) < INFINITY; }
// (Sums in another order may round a score up past lse, by a step that is not
// small here.)  A NaN stays.
__device__ __forceinline__ float at_most_0(float x) { return x > 0.0f ? 0.0f : x; }

template <class T>
__device__ __noinline__ float sum_again(const Attention &a, int32_t b, int32_t head, int32_t i, int32_t pos, int32_t visible,
                                        float lse)
{
    const T *q = static_cast<const T *>(a.q) + b * a.qs.batch + i * a.qs.len + head * a.qs.head;
    const T *k = static_cast<const T *>(a.k) + b * a.ks.batch + head / a.group * a.ks.head;
    float sum = 0.0f;
#pragma unroll 1
    for (int32_t j = 0; j < visible; ++j, k += a.ks.len) {
        float dot = 0.0f;
#pragma unroll 4
        for (int32_t d = 0; d < a.dim; d += 8) {
            float u[8], v[8];
            unpack<T, 8>(load<false, T, 8>(q + d), u);
            unpack<T, 8>(load<false, T, 8>(k + d), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = fmaf(u[e], v[e], dot);
        }
        const float bias = to_f32(static_cast<const T *>(a.table)[bucket_of(a.buckets, static_cast<int64_t>(j) - pos) * a.heads + head]);
        sum += exp2_approx(at_most_0(fmaf(dot, a.scale, bias) - lse) * kLog2e);
    }
    return sum;
}

// The bias added to N scaled scores whose relative positions descend from that
// of `at`: from the table by relative position, or one value beyond the last
// bucket's start on either side.
template <int N>
__device__ __forceinline__ void add_bias(uint32_t (&s)[N], float scale, const float *table, int32_t at, bool far, float edge)
{
    const float2 k2 = make_float2(scale, scale);
    if (far) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 f = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), k2, make_float2(edge, edge));
            s[e] = __float_as_uint(f.x), s[e + 1] = __float_as_uint(f.y);
        }
    } else {
        const float *t = table + at;
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 f = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), k2, make_float2(t[-e], t[-e - 1]));
            s[e] = __float_as_uint(f.x), s[e + 1] = __float_as_uint(f.y);
        }
    }
}

// ---- dq ------------------------------------------------------------------------

// Sums along the diagonals of a warp's 32 x 32 pairs are walked in that many
// parts of the columns at once: a step waits for a shuffle (16 x 1024 of 16
// heads of 64, 32 buckets: 519 us with two, 525 with one, 521 with four).
constexpr int kWalks = 2;

template <int kDim>
struct QueryShape {
    using Team = Crew<3, 1>;
    static constexpr int kChains = 3;
    static constexpr int kBoxes = kDim / 64;
    static constexpr uint32_t kRowsBytes = kBoxes * kRowsBox, kColsBytes = kBoxes * kColsBox;
    static constexpr int kStages = kDim == 64 ? 8 : 4;
    static constexpr uint32_t kStageBytes = 2 * kColsBytes;  // k, v
    static constexpr uint32_t kRing = 2 * kRowsBytes;        // after q, do
    static constexpr uint32_t kTable = kRing + kStages * kStageBytes;
};

struct QueryItem {
    int32_t b, pack, head0, head_kv, q_tile, i0, keys, pos0, tiles;
};

__device__ __forceinline__ QueryItem query_item(const BwdParams &p, uint32_t x)
{
    const Attention &a = p.a;
    QueryItem w;
    int32_t unit;
    if (a.causal) {  // the longest first
        p.by_units.divide(x, w.q_tile, unit);
        w.q_tile = p.q_tiles - 1 - w.q_tile;
    } else {
        p.by_q_tiles.divide(x, unit, w.q_tile);
    }
    const int32_t rows_per = kRows >> p.pack_log;
    p.by_packs.divide(unit, w.b, w.pack);
    w.head0 = w.pack << p.pack_log, w.head_kv = p.by_group.quotient(w.head0);
    w.i0 = w.q_tile * rows_per;
    w.keys = uniform(keys_of(a, w.b)), w.pos0 = first_position(a, w.keys);
    const int32_t last = min(w.i0 + rows_per, a.len_q) - 1, end = a.causal ? min(w.keys, w.pos0 + last + 1) : w.keys;
    w.tiles = max(0, (end + kCols - 1) / kCols);
    return w;
}

template <class T, int kDim, bool kDrop, bool kBias, bool kTwoTerms>
__global__ void __launch_bounds__(QueryShape<kDim>::Team::kThreads, 1) query_kernel(const __grid_constant__ BwdParams p)
{
    using S = QueryShape<kDim>;
    using Team = typename S::Team;
    constexpr int kChains = S::kChains;
    extern __shared__ uint8_t dynamic[];
    __shared__ alignas(16) uint4 response;
    __shared__ alignas(8) uint64_t bars[2 * S::kStages + 2 * kChains + 7];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t stalled;
    __shared__ float deltas[kChains][kRows];
    __shared__ float diagonals[kBias ? 4 * kChains : 1][kWalks][64], by_bucket[kBias ? 4 * kChains : 1][kMaxBuckets];
    const Attention &a = p.a;
    const uint32_t warp = uniform(threadIdx.x / 32u), lane = threadIdx.x % 32u;
    uint8_t *smem = dynamic + ((1024u - (smem_address(dynamic) & 1023u)) & 1023u);
    const uint32_t base = smem_address(smem);
    float *table = reinterpret_cast<float *>(smem + S::kTable);

    const uint32_t full = smem_address(bars), empty = full + 8 * S::kStages, scored = empty + 8 * S::kStages,
                   ready = scored + 8 * kChains, done = ready + 8 * kChains, q_full = done + 8, q_empty = q_full + 8,
                   tail = q_empty + 8, answered = tail + 8, heard = answered + 8, drained = heard + 8;
    if (threadIdx.x == 0) {
        prefetch_map(&p.q_rows), prefetch_map(&p.do_rows), prefetch_map(&p.k_cols), prefetch_map(&p.v_cols);
        stalled = 0;
        for (int s = 0; s < S::kStages; ++s) barrier_init(full + 8 * s, 1), barrier_init(empty + 8 * s, 1);
        for (int s = 0; s < kChains; ++s) barrier_init(scored + 8 * s, 1), barrier_init(ready + 8 * s, 4);
        barrier_init(done, 1), barrier_init(q_full, 1), barrier_init(q_empty, 1), barrier_init(tail, 1);
        barrier_init(answered, 1), barrier_init(heard, 1 + 4 * kChains), barrier_init(drained, 1);
        fence_barrier_init();
    }
    if (warp == Team::kMmaWarp) tmem_alloc<512>(smem_address(&tmem_base));
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base, scores_at = tmem + kDim;  // dq, then kChains times S and dP
    WorkQueue work{smem_address(&response), answered, heard, &stalled};
    if (warp >= Team::kTmaWarp) {
        give_registers<Team::kOtherRegisters>();
        if (warp == Team::kTmaWarp) {
            // ---- TMA: q and do, then K_n and V_n
            uint32_t use = 0, loaded = 0, tails = 0;
            bool fine = true;
            for (int32_t x = blockIdx.x; x >= 0; x = fine ? work.ask_warp() : -1) {
                const QueryItem w = query_item(p, x);
                if (!w.tiles) continue;
                if (loaded) fine = barrier_wait(q_empty, (loaded - 1) & 1u, &stalled);
                if (!fine) break;
                ++loaded;
                if (elect_one()) {
                    barrier_expect(q_full, 2 * S::kRowsBytes);
                    for (int c = 0; c < S::kBoxes; ++c) {
                        tma_load_5d(base + c * kRowsBox, &p.q_rows, q_full, c * 64, 0, w.i0, w.pack, w.b);
                        tma_load_5d(base + S::kRowsBytes + c * kRowsBox, &p.do_rows, q_full, c * 64, 0, w.i0, w.pack, w.b);
                    }
                }
#pragma unroll 1
                for (int32_t n = 0; n < w.tiles; ++n) {
                    const int32_t j0 = n * kCols;
                    const uint32_t stage = use % S::kStages, bar = full + 8 * stage, dst = base + S::kRing + stage * S::kStageBytes;
                    fine = barrier_wait(empty + 8 * stage, (use / S::kStages & 1u) ^ 1u, &stalled);
                    if (!fine) break;
                    ++use;
                    // keys past n(b) that the array holds: whatever they are, dS's zeros must meet zeros
                    const bool past = j0 + kCols > w.keys && w.keys < a.len_k;
                    const uint32_t on = past ? tail : bar;
                    if (elect_one()) {
                        barrier_expect(on, S::kStageBytes);
                        for (int c = 0; c < S::kBoxes; ++c) {
                            tma_load_5d(dst + c * kColsBox, &p.k_cols, on, c * 64, 0, j0, w.head_kv, w.b);
                            tma_load_5d(dst + S::kColsBytes + c * kColsBox, &p.v_cols, on, c * 64, 0, j0, w.head_kv, w.b);
                        }
                    }
                    if (past) {
                        if (!barrier_wait(tail, tails++ & 1u, &stalled)) barrier_drain(tail, (tails - 1) & 1u);
                        uint8_t *rows = smem + S::kRing + stage * S::kStageBytes;
                        for (int c = 0; c < S::kBoxes; ++c)
#pragma unroll 1
                            for (uint32_t o = (w.keys - j0) * 128u + lane * 16u; o < kColsBox; o += 512u)
                                *reinterpret_cast<uint4 *>(rows + c * kColsBox + o) = make_uint4(0, 0, 0, 0);
                        fence_async_shared();
                        __syncwarp();
                        if (elect_one()) barrier_arrive(bar);
                    }
                }
            }
            if (stalled) {  // nothing may land after the block has ended
                if (loaded) barrier_drain(q_full, (loaded - 1) & 1u);
                for (uint32_t u = use > S::kStages ? use - S::kStages : 0; u < use; ++u) barrier_drain(full + 8 * (u % S::kStages), u / S::kStages & 1u);
            }
        } else if (warp == Team::kMmaWarp) {
            // ---- MMA
            constexpr uint32_t kScores = mma_shape<T>(kCols, false), kOut = mma_shape<T>(kDim, true);
            const uint64_t qd = row_major_tile(base), dd = row_major_tile(base + S::kRowsBytes);
            const uint64_t ring_k = row_major_tile(base + S::kRing), ring_v = row_major_tile(base + S::kRing + S::kColsBytes);
            const uint64_t ring_kt = column_major_tile(base + S::kRing, S::kBoxes > 1 ? kColsBox : 1024);
            // tile counters over all items: made is kChains ahead of added within an item
            uint32_t use_made = 0, use_added = 0, loaded = 0, turns = 0;  // turns: bit c, the parity of chain c's next dS
            bool fine = true;
            for (int32_t x = blockIdx.x; x >= 0; x = fine ? work.next_warp() : -1) {
                const int32_t tiles = query_item(p, x).tiles;
                if (!tiles) continue;
                fine = barrier_wait(q_full, loaded++ & 1u, &stalled);
                uint32_t chain = 0;
#pragma unroll 1
                for (int32_t n = -kChains; n < tiles && fine; ++n) {
                    const bool add = n >= 0, make = n + kChains < tiles;
                    const uint32_t at = scores_at + chain * 2 * kCols, stage = use_added % S::kStages, next = use_made % S::kStages;
                    if (add) fine = barrier_wait(ready + 8 * chain, turns >> chain & 1u, &stalled);
                    if (!fine) break;
                    tmem_fence_after();
                    if (add && elect_one()) {  // dQ += dS K
                        const uint64_t kd = ring_kt + stage * (S::kStageBytes / 16);
#pragma unroll
                        for (int i = 0; i < kCols / 16; ++i) mma_step_tmem(tmem, at + i * 8, kd + i * (2048 / 16), kOut, n > 0 || i > 0);
                        if (kTwoTerms)
#pragma unroll
                            for (int i = 0; i < kCols / 16; ++i) mma_step_tmem(tmem, at + kCols + i * 8, kd + i * (2048 / 16), kOut, true);
                        mma_commit(empty + 8 * stage);
                        if (n + 1 == tiles) mma_commit(done);
                    }
                    if (make) fine = barrier_wait(full + 8 * next, use_made / S::kStages & 1u, &stalled);
                    if (!fine) break;
                    tmem_fence_after();
                    if (make && elect_one()) {  // S = Q K^T, dP = dO V^T
                        const uint64_t kd = ring_k + next * (S::kStageBytes / 16), vd = ring_v + next * (S::kStageBytes / 16);
#pragma unroll
                        for (int i = 0; i < kDim / 16; ++i) mma_step(at, qd + row_step(i, kRowsBox), kd + row_step(i, kColsBox), kScores, i > 0);
#pragma unroll
                        for (int i = 0; i < kDim / 16; ++i)
                            mma_step(at + kCols, dd + row_step(i, kRowsBox), vd + row_step(i, kColsBox), kScores, i > 0);
                        mma_commit(scored + 8 * chain);
                        if (n + kChains + 1 == tiles) mma_commit(q_empty);
                    }
                    __syncwarp();
                    if (add) ++use_added, turns ^= 1u << chain;
                    use_made += make;
                    chain = chain + 1 == kChains ? 0 : chain + 1;
                }
            }
            if (stalled && elect_one()) mma_commit(drained), barrier_drain(drained, 0);
        }
    } else {
        take_registers<Team::kWorkerRegisters>();
        // ---- the rows: a query to a thread, a chain to a warpgroup
        const uint32_t chain = warp / 4;
        const int32_t r = (warp % 4) * 32 + lane;
        const uint32_t lanes = (warp % 4) * 32u << 16;
        const uint32_t mine = scores_at + lanes + chain * 2 * kCols;  // S, then dS; dP kCols on
        const int32_t reach = bias_reach(a.buckets);
        const int32_t last_start = kBias ? a.buckets.starts[a.buckets.count - 2] : 0;
        int32_t table_head = -1;
        // the bucket of every relative position that is tabulated (read after the item's first barrier)
        uint8_t *bucket_at = reinterpret_cast<uint8_t *>(table + 2 * reach) + reach;
        if (kBias)
            for (int32_t t = threadIdx.x; t < 2 * reach; t += Team::kWorkers) bucket_at[t - reach] = bucket_of(a.buckets, t - reach);
        if (kBias) {  // the diagonals that a walk does not reach stay 0
            for (int k = 0; k < kWalks; ++k) diagonals[warp][k][lane] = diagonals[warp][k][lane + 32] = 0.0f;
            __syncwarp();
        }
        uint32_t turn = 0, finished = 0;
        // A row's o, do (the warpgroups take parts of it) and lse are asked for before the previous item's result is
        // written, which takes longer than they do.
        constexpr int kParts = (kDim / 8 + kChains - 1) / kChains;
        Raw<T, 8> part_o[kParts], part_do[kParts];
        float next_lse;
        auto fetch_row = [&](const QueryItem &w) {
            const int32_t i = min(w.i0 + (r >> p.pack_log), a.len_q - 1), head = w.head0 + (r & (p.pack - 1));
            const T *o = static_cast<const T *>(a.o) + w.b * a.os.batch + i * a.os.len + head * a.os.head;
            const T *d_o = static_cast<const T *>(a.d_o) + w.b * a.dos.batch + i * a.dos.len + head * a.dos.head;
#pragma unroll
            for (int k = 0; k < kParts; ++k) {
                const int32_t at = min(8 * (k * kChains + static_cast<int32_t>(chain)), a.dim - 8);
                part_o[k] = load<false, T, 8>(o + at), part_do[k] = load<false, T, 8>(d_o + at);
            }
            next_lse = a.lse[(static_cast<int64_t>(w.b) * a.heads + head) * a.len_q + i];
        };
        QueryItem w = query_item(p, blockIdx.x);
        fetch_row(w);
        for (;;) {
            const int32_t warp_i = w.i0 + ((warp % 4) * 32 >> p.pack_log);
            const int32_t i = w.i0 + (r >> p.pack_log), head = w.head0 + (r & (p.pack - 1)), pos = w.pos0 + i;
            const bool valid = i < a.len_q, any = warp_i < a.len_q;
            const int64_t index = static_cast<int64_t>(w.b) * a.heads + head;
            const uint32_t counter = a.first + (static_cast<uint32_t>(index) * a.len_q + i) * static_cast<uint32_t>(a.len_k);
            const int32_t visible = a.causal ? min(w.keys, pos + 1) : w.keys;
            const int32_t warp_visible = a.causal ? min(w.keys, w.pos0 + warp_i + 1) : w.keys;

            // lse and delta = sum of o do
            float lse = INFINITY, delta = 0.0f;
            if (valid) {
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    if (8 * (k * kChains + static_cast<int32_t>(chain)) < a.dim) {
                        float u[8], v[8];
                        unpack<T, 8>(part_o[k], u);
                        unpack<T, 8>(part_do[k], v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) delta += u[e] * v[e];
                    }
                }
                // a query that sees nothing: exp(s - inf) = 0 whatever its scores
                lse = next_lse == -INFINITY ? INFINITY : kBias ? next_lse : next_lse * kLog2e;
            }
            deltas[chain][r] = delta;
            sync_threads<Team::kWorkers>(1);
            delta = 0.0f;
#pragma unroll
            for (int c = 0; c < kChains; ++c) delta += deltas[c][r];
            const float minus_delta = -delta;
            float share = a.mask.scale, to_key = kBias ? -lse : kLift<T> - lse;
            bool some = false;  // of the warp's queries have too large an lse
            if constexpr (kMayLose<T, kBias>) {
                const bool lost = valid && loses(next_lse);
                some = __any_sync(0xFFFFFFFFu, lost);
                if (lost) {
                    const float sum = sum_again<T>(a, w.b, head, i, pos, visible, lse);
                    share /= sum, delta /= sum, to_key = -logf(sum);
                }
                if (chain == 0 && lane == 0 && warp_i < p.len_pad) p.lost[index * (p.len_pad / 32) + warp_i / 32] = some;
            }
            if (valid && chain == 0) p.stats[index * p.len_pad + i] = make_float2(to_key, minus_delta * kUnlift<T>);
            if (w.q_tile == p.q_tiles - 1)  // what key_kernel reads past the last query
                for (int32_t t = threadIdx.x; t < p.pack * (p.len_pad - a.len_q); t += Team::kWorkers)
                    p.stats[(static_cast<int64_t>(w.b) * a.heads + w.head0 + (t & (p.pack - 1))) * p.len_pad + a.len_q + (t >> p.pack_log)] =
                        make_float2(-INFINITY, 0.0f);
            if (kBias && w.head0 != table_head) {  // the bias by relative position (pack is 1)
                table_head = w.head0;
                for (int32_t t = threadIdx.x; t < 2 * reach; t += Team::kWorkers)
                    table[t] = to_f32(static_cast<const T *>(a.table)[bucket_of(a.buckets, t - reach) * a.heads + w.head0]);
                sync_threads<Team::kWorkers>(1);
            }
            if (kBias && w.b == 0 && w.q_tile == 0)
                for (int32_t t = threadIdx.x; t < 2 * reach; t += Team::kWorkers)
                    p.bias[static_cast<int64_t>(w.head0) * 2 * reach + t] = table[t];

            float far_low = 0.0f, far_high = 0.0f;
            if (kBias && a.dtable) {
                for (uint32_t m = lane; m < kMaxBuckets; m += 32) by_bucket[warp][m] = 0.0f;
                __syncwarp();
            }
            auto tiles = [&](auto lose) {
                const float of_dp = decltype(lose)::value ? share : a.mask.scale;
                const float2 scale = make_float2(of_dp, of_dp), minus = make_float2(-delta, -delta);
#pragma unroll 1
                for (int32_t n = chain; n < w.tiles; n += kChains, ++turn) {
                    barrier_wait(scored + 8 * chain, turn & 1u, &stalled);
                    tmem_fence_after();
                    if (any) {
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            const int32_t j0 = n * kCols + 32 * c;
                            uint32_t s[32], dp[32];
                            tmem_load(s, mine + 32 * c);
                            tmem_load(dp, mine + kCols + 32 * c);
                            tmem_wait_load(s, dp);
                            const int32_t low = j0 - (w.pos0 + warp_i + 31), high = j0 + 31 - (w.pos0 + warp_i);
                            const bool far = high <= -last_start || low >= last_start;
                            // the exponential's argument in base two is s by + at: of the score, with one bias for all pairs,
                            // or of what has become of it.  A bias as large as a type's lowest value leaves nothing of s.
                            float by = a.scale * kLog2e, at = -lse;
                            if constexpr (decltype(lose)::value) {
                                const float edge = table[high < 0 ? 0 : 2 * reach - 1], *t = table + (j0 - pos + reach);
                                by = kLog2e, at = 0.0f;
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    s[e] = __float_as_uint(at_most_0(fmaf(__uint_as_float(s[e]), a.scale, far ? edge : t[e]) - lse));
                            } else if (kBias && far) {
                                const float edge = table[high < 0 ? 0 : 2 * reach - 1];
                                by = fabsf(edge) < 0x1p100f ? by : 0.0f, at = (edge - lse) * kLog2e;
                            } else if (kBias) {
                                by = 1.0f, at = 0.0f;
                                const float *t = table + (j0 - pos + reach);
                                const float2 scale = make_float2(a.scale, a.scale), from = make_float2(-lse, -lse), b2 = make_float2(kLog2e, kLog2e);
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    float2 f = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                                    f = mul2(add2(fma2(f, scale, make_float2(t[e], t[e + 1])), from), b2);
                                    s[e] = __float_as_uint(f.x), s[e + 1] = __float_as_uint(f.y);
                                }
                            }
                            const float2 by2 = make_float2(by, by), at2 = make_float2(at, at);
                            // P = exp(S - lse); dS = P (dP / (1 - p) - delta), dP dropped as P was
                            for_pairs32<kDrop>(a.mask, counter + j0, [&](uint32_t e, float2 k) {
                                float2 f = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                                f = fma2(f, by2, at2);
                                const float2 prob = make_float2(exp2_approx(f.x), exp2_approx(f.y));
                                float2 d = make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1]));
                                if (kDrop) d = mul2(d, k);
                                d = mul2(fma2(d, scale, minus), prob);
                                s[e] = __float_as_uint(d.x), s[e + 1] = __float_as_uint(d.y);
                            });
                            if (j0 + 32 > warp_visible) {
                                const int32_t seen = visible - j0;
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (e >= seen) s[e] = 0;
                            }
                            uint32_t ds[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) ds[e] = pack2<T>(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
                            tmem_store(mine + 16 * c, ds);
                            if (kTwoTerms) {  // the second, over dP
                                uint32_t rest[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    rest[e] = rest2<T>(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), ds[e]);
                                tmem_store(mine + kCols + 16 * c, rest);
                            }
                            if (c) {
                                tmem_wait_store();
                                tmem_fence_before();
                                __syncwarp();
                                if (lane == 0) barrier_arrive(ready + 8 * chain);
                            }
                            if (kBias && a.dtable) {
                                if (far) {  // one bucket
                                    float2 total = make_float2(0.0f, 0.0f);
#pragma unroll
                                    for (int e = 0; e < 32; e += 2) total = add2(total, make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])));
                                    (high <= -last_start ? far_low : far_high) += total.x + total.y;
                                } else {
                                    // Sums along the diagonals of the warp's 32 x 32 pairs: a partial sum moves one row down
                                    // with each column; what leaves row 31, or is left in a walk's last column, is a walk's
                                    // part.  Diagonal d = 0 .. 62 is relative position low + d.
                                    constexpr int kSteps = 32 / kWalks;
                                    float acc[kWalks] = {};
#pragma unroll
                                    for (int e = 0; e < kSteps; ++e)
#pragma unroll
                                        for (int k = 0; k < kWalks; ++k) {
                                            const float before = __shfl_up_sync(0xFFFFFFFFu, acc[k], 1);
                                            acc[k] = (lane ? before : 0.0f) + __uint_as_float(s[k * kSteps + e]);
                                            if (lane == 31) diagonals[warp][k][k * kSteps + e] = acc[k];
                                        }
#pragma unroll
                                    for (int k = 0; k < kWalks; ++k)
                                        if (lane < 31) diagonals[warp][k][(k + 1) * kSteps + 30 - lane] = acc[k];
                                    __syncwarp();
                                    // A bucket's positions follow each other, so sums over runs of one bucket: half of the
                                    // diagonals at a time, the last lane of a run adds it.
                                    int32_t bucket[2];
                                    float run[2] = {};
#pragma unroll
                                    for (int d = 0; d < 2; ++d) {
                                        bucket[d] = bucket_at[low + 32 * d + lane];
#pragma unroll
                                        for (int k = 0; k < kWalks; ++k) run[d] += diagonals[warp][k][32 * d + lane];
                                    }
#pragma unroll
                                    for (int m = 1; m < 32; m *= 2)
#pragma unroll
                                        for (int d = 0; d < 2; ++d) {
                                            const float before = __shfl_up_sync(0xFFFFFFFFu, run[d], m);
                                            const int32_t its = __shfl_up_sync(0xFFFFFFFFu, bucket[d], m);
                                            if (static_cast<int>(lane) >= m && its == bucket[d]) run[d] += before;
                                        }
#pragma unroll
                                    for (int d = 0; d < 2; ++d) {
                                        const int32_t after = __shfl_down_sync(0xFFFFFFFFu, bucket[d], 1);
                                        if (lane == 31 || after != bucket[d]) by_bucket[warp][bucket[d]] += run[d];
                                        __syncwarp();
                                    }
                                }
                            }
                        }
                    } else if (lane == 0) {
                        barrier_arrive(ready + 8 * chain);
                    }
                }
            };
            if (!some) tiles(std::false_type{});
            else tiles(std::true_type{});

            // ---- the next item, and this one's result
            const int32_t x = work.next_warp();
            QueryItem next = w;
            if (x >= 0) {
                next = query_item(p, x);
                fetch_row(next);
            }
            if (kBias && a.dtable) {
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) {
                    far_low += __shfl_xor_sync(0xFFFFFFFFu, far_low, m);
                    far_high += __shfl_xor_sync(0xFFFFFFFFu, far_high, m);
                }
                if (lane == 0) {
                    by_bucket[warp][a.buckets.count - 1] += far_low;
                    by_bucket[warp][a.buckets.past ? a.buckets.total - 1 : 0] += far_high;
                }
                sync_threads<Team::kWorkers>(1);
                if (threadIdx.x < a.buckets.total) {
                    float s = 0.0f;
                    for (int k = 0; k < 4 * kChains; ++k) s += by_bucket[k][threadIdx.x];
                    p.sums[((static_cast<int64_t>(w.b) * a.heads + w.head0) * p.q_tiles + w.q_tile) * a.buckets.total + threadIdx.x] = s;
                }
            }
            if (w.tiles) {
                barrier_wait(done, finished++ & 1u, &stalled);
                tmem_fence_after();
            }
            if (any && chain < 2) {  // two warpgroups write half of the columns each
                T *row = static_cast<T *>(a.dq) + w.b * a.dqs.batch + i * a.dqs.len + head * a.dqs.head;
#pragma unroll 1
                for (int c = 0; c < kDim / 64; ++c) {
                    uint32_t o[32] = {};
                    const int col = chain * (kDim / 2) + 32 * c;
                    if (w.tiles) {
                        tmem_load(o, tmem + lanes + col);
                        tmem_wait_load(o);
                    }
                    if (valid) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float eight[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) eight[k] = __uint_as_float(o[e + k]) * a.scale;
                            if (col + e < a.dim) store<T, 8>(row + col + e, eight);
                        }
                    }
                }
            }
            // dq has been read before the next item's first dS is announced; and all leave together, also when a
            // wait of one of them ran out
            tmem_fence_before();
            if (!all_of<Team::kWorkers>(1, x >= 0)) break;
            w = next;
        }
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == Team::kMmaWarp) tmem_free<512>(tmem);
}

// ---- dk, dv ----------------------------------------------------------------------

template <int kDim>
struct KeyShape {
    static constexpr int kChains = kDim == 64 ? 3 : 2, kShare = kDim == 64 ? 1 : 2;
    using Team = Crew<kChains, kShare>;
    static constexpr int kBoxes = kDim / 64;
    static constexpr uint32_t kRowsBytes = kBoxes * kRowsBox, kColsBytes = kBoxes * kColsBox;
    static constexpr int kStages = kDim == 64 ? 8 : 4;
    static constexpr uint32_t kStageBytes = 2 * kColsBytes;            // q, do
    static constexpr uint32_t kRing = 2 * kRowsBytes;                  // after k, v
    static constexpr uint32_t kStats = kRing + kStages * kStageBytes;  // kCols (lse, delta) a stage
    static constexpr uint32_t kBytes = kStats + kStages * kCols * sizeof(float2);
    // where a thread's 16 columns of 16-bit pairs are for its 32 columns of S: packed from the front by one warpgroup,
    // each over its own half by two
    static constexpr uint32_t kPitch = kShare == 1 ? 16 : 32;
};

struct KeyItem {
    int32_t b, head_kv, j0, keys, pos0, begin, per_head, tiles;
};

// The first query that sees any of the keys from j0 on.
__device__ __forceinline__ int32_t first_query(const Attention &a, int32_t j0, int32_t pos0)
{
    return a.causal && j0 > pos0 ? j0 - pos0 : 0;
}

__device__ __forceinline__ KeyItem key_item(const BwdParams &p, uint32_t x)
{
    const Attention &a = p.a;
    KeyItem w;
    int32_t tile, unit;
    p.by_key_units.divide(x, tile, unit);  // the first keys, whose causal part is the longest, first
    p.by_heads_kv.divide(unit, w.b, w.head_kv);
    w.j0 = tile * kRows;
    w.keys = uniform(keys_of(a, w.b)), w.pos0 = first_position(a, w.keys);
    const int32_t q_tiles = (a.len_q + kCols - 1) / kCols;
    w.begin = min(first_query(a, w.j0, w.pos0) / kCols, q_tiles), w.per_head = w.j0 < w.keys ? q_tiles - w.begin : 0;
    w.tiles = w.per_head * a.group;
    return w;
}

template <class T, int kDim, bool kDrop, bool kBias, bool kTwoTerms>
__global__ void __launch_bounds__(KeyShape<kDim>::Team::kThreads, 1) key_kernel(const __grid_constant__ BwdParams p)
{
    using S = KeyShape<kDim>;
    using Team = typename S::Team;
    constexpr int kChains = S::kChains;
    extern __shared__ uint8_t dynamic[];
    __shared__ alignas(16) uint4 response;
    __shared__ alignas(8) uint64_t bars[2 * S::kStages + 2 * kChains + 7];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t stalled;
    const Attention &a = p.a;
    const uint32_t warp = uniform(threadIdx.x / 32u), lane = threadIdx.x % 32u;
    uint8_t *smem = dynamic + ((1024u - (smem_address(dynamic) & 1023u)) & 1023u);
    const uint32_t base = smem_address(smem);

    const uint32_t full = smem_address(bars), empty = full + 8 * S::kStages, scored = empty + 8 * S::kStages,
                   ready = scored + 8 * kChains, done = ready + 8 * kChains, k_full = done + 8, k_empty = k_full + 8,
                   answered = k_empty + 8, heard = answered + 8, drained = heard + 8, tail = drained + 8;
    if (threadIdx.x == 0) {
        prefetch_map(&p.k_rows), prefetch_map(&p.v_rows), prefetch_map(&p.q_cols), prefetch_map(&p.do_cols);
        stalled = 0;
        for (int s = 0; s < S::kStages; ++s) barrier_init(full + 8 * s, 1), barrier_init(empty + 8 * s, 1);
        for (int s = 0; s < kChains; ++s) barrier_init(scored + 8 * s, 1), barrier_init(ready + 8 * s, 4 * S::kShare);
        barrier_init(done, 1), barrier_init(k_full, 1), barrier_init(k_empty, 1);
        barrier_init(answered, 1), barrier_init(heard, 1 + 4 * Team::kGroups), barrier_init(drained, 1), barrier_init(tail, 1);
        fence_barrier_init();
    }
    if (warp == Team::kMmaWarp) tmem_alloc<512>(smem_address(&tmem_base));
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base, dv_at = tmem, dk_at = tmem + kDim, scores_at = tmem + 2 * kDim;
    WorkQueue work{smem_address(&response), answered, heard, &stalled};
    if (warp >= Team::kTmaWarp) {
        give_registers<Team::kOtherRegisters>();
        if (warp == Team::kTmaWarp) {
            // ---- TMA: k and v, then the queries' tiles, head by head
            uint32_t use = 0, loaded = 0, tails = 0;
            bool fine = true;
            for (int32_t x = blockIdx.x; x >= 0; x = fine ? work.ask_warp() : -1) {
                const KeyItem w = key_item(p, x);
                if (!w.tiles) continue;
                if (loaded) fine = barrier_wait(k_empty, (loaded - 1) & 1u, &stalled);
                if (!fine) break;
                ++loaded;
                if (elect_one()) {
                    barrier_expect(k_full, 2 * S::kRowsBytes);
                    for (int c = 0; c < S::kBoxes; ++c) {
                        tma_load_5d(base + c * kRowsBox, &p.k_rows, k_full, c * 64, 0, w.j0, w.head_kv, w.b);
                        tma_load_5d(base + S::kRowsBytes + c * kRowsBox, &p.v_rows, k_full, c * 64, 0, w.j0, w.head_kv, w.b);
                    }
                }
                // Queries of the first tile that see none of the keys (before the first key, perhaps, where what q and
                // do hold is nobody's gradient): whatever they are, the zeros of P and dS must meet zeros.
                const uint32_t hidden = first_query(a, w.j0, w.pos0) % kCols;
                int32_t head = w.head_kv * a.group, t = w.begin;
#pragma unroll 1
                for (int32_t n = 0; n < w.tiles; ++n) {
                    const uint32_t stage = use % S::kStages, bar = full + 8 * stage, dst = base + S::kRing + stage * S::kStageBytes;
                    fine = barrier_wait(empty + 8 * stage, (use / S::kStages & 1u) ^ 1u, &stalled);
                    if (!fine) break;
                    ++use;
                    const bool clears = hidden > 0 && t == w.begin;
                    const uint32_t on = clears ? tail : bar;
                    if (elect_one()) {
                        barrier_expect(on, S::kStageBytes + kCols * sizeof(float2));
                        for (int c = 0; c < S::kBoxes; ++c) {
                            tma_load_5d(dst + c * kColsBox, &p.q_cols, on, c * 64, 0, t * kCols, head, w.b);
                            tma_load_5d(dst + S::kColsBytes + c * kColsBox, &p.do_cols, on, c * 64, 0, t * kCols, head, w.b);
                        }
                        bulk_load(base + S::kStats + stage * kCols * sizeof(float2),
                                  p.stats + (static_cast<int64_t>(w.b) * a.heads + head) * p.len_pad + t * kCols, kCols * sizeof(float2), on);
                    }
                    if (clears) {
                        if (!barrier_wait(tail, tails++ & 1u, &stalled)) barrier_drain(tail, (tails - 1) & 1u);
                        uint8_t *rows = smem + S::kRing + stage * S::kStageBytes;
#pragma unroll 1
                        for (int c = 0; c < 2 * S::kBoxes; ++c)  // q's, then do's
#pragma unroll 1
                            for (uint32_t o = lane * 16u; o < hidden * 128u; o += 512u)
                                *reinterpret_cast<uint4 *>(rows + c * kColsBox + o) = make_uint4(0, 0, 0, 0);
                        fence_async_shared();
                        __syncwarp();
                        if (elect_one()) barrier_arrive(bar);
                    }
                    if (++t == w.begin + w.per_head) t = w.begin, ++head;
                }
            }
            if (stalled && elect_one()) {  // nothing may land after the block has ended
                if (loaded) barrier_drain(k_full, (loaded - 1) & 1u);
                for (uint32_t u = use > S::kStages ? use - S::kStages : 0; u < use; ++u)
                    barrier_drain(full + 8 * (u % S::kStages), u / S::kStages & 1u);
            }
        } else if (warp == Team::kMmaWarp) {
            // ---- MMA
            constexpr uint32_t kScores = mma_shape<T>(kCols, false), kOut = mma_shape<T>(kDim, true);
            const uint64_t kd = row_major_tile(base), vd = row_major_tile(base + S::kRowsBytes);
            const uint64_t ring_q = row_major_tile(base + S::kRing), ring_do = row_major_tile(base + S::kRing + S::kColsBytes);
            const uint64_t ring_qt = column_major_tile(base + S::kRing, S::kBoxes > 1 ? kColsBox : 1024);
            uint32_t use_made = 0, use_added = 0, loaded = 0, turns = 0;  // turns: bit c, the parity of chain c's next P, dS
            bool fine = true;
            for (int32_t x = blockIdx.x; x >= 0; x = fine ? work.next_warp() : -1) {
                const int32_t tiles = key_item(p, x).tiles;
                if (!tiles) continue;
                fine = barrier_wait(k_full, loaded++ & 1u, &stalled);
                uint32_t chain = 0;
#pragma unroll 1
                for (int32_t n = -kChains; n < tiles && fine; ++n) {
                    const bool add = n >= 0, make = n + kChains < tiles;
                    const uint32_t at = scores_at + chain * 2 * kCols, stage = use_added % S::kStages, next = use_made % S::kStages;
                    if (add) fine = barrier_wait(ready + 8 * chain, turns >> chain & 1u, &stalled);
                    if (!fine) break;
                    tmem_fence_after();
                    if (add && elect_one()) {  // dV += P^T dO, dK += dS^T Q
                        const uint64_t qt = ring_qt + stage * (S::kStageBytes / 16);
#pragma unroll
                        for (int i = 0; i < kCols / 16; ++i) {
                            const uint32_t from = kTwoTerms ? i * 16 : i / 2 * S::kPitch + i % 2 * 8;
                            mma_step_tmem(dv_at, at + from, qt + (S::kColsBytes + i * 2048) / 16, kOut, n > 0 || i > 0);
                            if (kTwoTerms) mma_step_tmem(dv_at, at + from + 8, qt + (S::kColsBytes + i * 2048) / 16, kOut, true);
                        }
#pragma unroll
                        for (int i = 0; i < kCols / 16; ++i) {
                            const uint32_t from = kCols + (kTwoTerms ? i * 16 : i / 2 * S::kPitch + i % 2 * 8);
                            mma_step_tmem(dk_at, at + from, qt + i * 2048 / 16, kOut, n > 0 || i > 0);
                            if (kTwoTerms) mma_step_tmem(dk_at, at + from + 8, qt + i * 2048 / 16, kOut, true);
                        }
                        mma_commit(empty + 8 * stage);
                        if (n + 1 == tiles) mma_commit(done);
                    }
                    if (make) fine = barrier_wait(full + 8 * next, use_made / S::kStages & 1u, &stalled);
                    if (!fine) break;
                    tmem_fence_after();
                    if (make && elect_one()) {  // S^T = K Q^T, dP^T = V dO^T
                        const uint64_t qd = ring_q + next * (S::kStageBytes / 16), dd = ring_do + next * (S::kStageBytes / 16);
#pragma unroll
                        for (int i = 0; i < kDim / 16; ++i) mma_step(at, kd + row_step(i, kRowsBox), qd + row_step(i, kColsBox), kScores, i > 0);
#pragma unroll
                        for (int i = 0; i < kDim / 16; ++i)
                            mma_step(at + kCols, vd + row_step(i, kRowsBox), dd + row_step(i, kColsBox), kScores, i > 0);
                        mma_commit(scored + 8 * chain);
                        if (n + kChains + 1 == tiles) mma_commit(k_empty);
                    }
                    __syncwarp();
                    if (add) ++use_added, turns ^= 1u << chain;
                    use_made += make;
                    chain = chain + 1 == kChains ? 0 : chain + 1;
                }
            }
            if (stalled && elect_one()) mma_commit(drained), barrier_drain(drained, 0);
        }
    } else {
        take_registers<Team::kWorkerRegisters>();
        // ---- the rows: a key to a thread, a chain to a warpgroup or two
        const uint32_t chain = warp / (4 * S::kShare), half = S::kShare == 1 ? 0 : warp / 4 % 2;
        const int32_t r = (warp % 4) * 32 + lane;
        const uint32_t lanes = (warp % 4) * 32u << 16;
        const uint32_t mine = scores_at + lanes + chain * 2 * kCols;  // S^T, then P^T; kCols on, dP^T, then dS^T
        const int32_t reach = bias_reach(a.buckets);
        const int32_t last_start = kBias ? a.buckets.starts[a.buckets.count - 2] : 0;
        const float scale = a.mask.scale * kUnlift<T>, to_base2 = a.scale * kLog2e;
        // Columns at a time: with 104 registers a thread, 32 of S and dP spill (2 x 4096 causal queries of 16 heads of
        // 128: 522 us with 16, 567 with 32); with 152, 16 only wait for TMEM more often (16 x 1024 of 16 heads of 64:
        // 577 us with 32, 611 with 16).
        constexpr int kPiece = S::kShare == 1 ? 32 : 16;
        uint32_t turn = 0, use = 0, finished = 0;
        // Whether queries of the item have too large an lse: asked for before the previous item's result is written,
        // which takes longer.  A lane's part of the answer.
        auto fetch_lost = [&](const KeyItem &w) {
            uint32_t any = 0;
            if constexpr (kMayLose<T, kBias>) {
                const int32_t words = p.len_pad / kCols * a.group;  // of two bytes, the heads' one after the other (a q of 2^31 would be 2 TB)
                const uint16_t *of_heads = reinterpret_cast<const uint16_t *>(p.lost) +
                                           (static_cast<int64_t>(w.b) * a.heads_kv + w.head_kv) * words;
#pragma unroll 1
                for (int32_t x = lane + 32; x < words; x += 32) any |= of_heads[x];
                if (lane < words) any |= of_heads[lane];
            }
            return any;
        };
        KeyItem w = key_item(p, blockIdx.x);
        uint32_t lost = fetch_lost(w);
        for (;;) {
            const int32_t j = w.j0 + r, warp_j = w.j0 + (warp % 4) * 32;
            const bool any = warp_j < w.keys;
            const bool some = kMayLose<T, kBias> && __any_sync(0xFFFFFFFFu, lost != 0u);
            auto tiles = [&](auto lose) {
                int32_t head = w.head_kv * a.group, t = chain;  // tile n is tile t of a head's
#pragma unroll 1
                for (int32_t n = chain; n < w.tiles; n += kChains, t += kChains, ++turn) {
                    while (t >= w.per_head) t -= w.per_head, ++head;
                    const int32_t i0 = (w.begin + t) * kCols;
                    const float4 *tile_stats = reinterpret_cast<const float4 *>(smem + S::kStats + (use + n) % S::kStages * kCols * sizeof(float2));
                    barrier_wait(scored + 8 * chain, turn & 1u, &stalled);
                    tmem_fence_after();
                    if (any) {
#pragma unroll 1
                        for (int at = half * kCols / S::kShare; at < (half + 1) * kCols / S::kShare; at += kPiece) {
                            const float4 *stats = tile_stats + at / 2;
                            uint32_t s[kPiece], dp[kPiece];  // S^T, dP^T
                            tmem_load(s, mine + at);
                            tmem_load(dp, mine + kCols + at);
                            tmem_wait_load(s, dp);
                            const int32_t ic = i0 + at, rel = j - w.pos0 - ic;  // to the first of kPiece queries
                            const int32_t low = warp_j - w.pos0 - ic - kPiece + 1, high = warp_j + 31 - w.pos0 - ic;
                            const uint32_t counter = a.first + ((static_cast<uint32_t>(w.b) * a.heads + head) * a.len_q + ic) * static_cast<uint32_t>(a.len_k) + j;
                            if (kBias) {
                                const float *bias = p.bias + static_cast<int64_t>(head) * 2 * reach;
                                const bool far = high <= -last_start || low >= last_start;
                                const float edge = far ? bias[high < 0 ? 0 : 2 * reach - 1] : 0.0f;
                                if constexpr (decltype(lose)::value) {
                                    const float *lse = a.lse + (static_cast<int64_t>(w.b) * a.heads + head) * a.len_q;
#pragma unroll
                                    for (int e = 0; e < kPiece; ++e) {
                                        const float x = fmaf(__uint_as_float(s[e]), a.scale, far ? edge : bias[rel + reach - e]);
                                        const float shift = lse[min(ic + e, a.len_q - 1)];
                                        s[e] = __float_as_uint(loses(shift) ? at_most_0(x - shift) : x);
                                    }
                                } else {
                                    add_bias(s, a.scale, bias, rel + reach, far, edge);
                                }
                            }
                            // P = exp(S - lse), dropped for dv; dS = P (dropout(dP) - delta) for dk
                            auto pair = [&](int e, float2 &kept2, float2 &d) {
                                const float4 st = stats[e / 2];  // two queries' -lse, -delta
                                float2 f = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                                f = kBias ? fma2(add2(f, make_float2(st.x, st.z)), make_float2(kLog2e, kLog2e), make_float2(kLift<T>, kLift<T>))
                                          : fma2(f, make_float2(to_base2, to_base2), make_float2(st.x, st.z));
                                const float2 prob = make_float2(exp2_approx(f.x), exp2_approx(f.y));
                                kept2 = prob, d = make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1]));
                                if (kDrop) {
                                    const uint32_t step = a.len_k;
                                    const float2 k = make_float2(kept(a.mask, mad_lo(e, step, counter)), kept(a.mask, mad_lo(e + 1, step, counter)));
                                    kept2 = mul2(kept2, k), d = mul2(d, k);
                                }
                                d = mul2(fma2(d, make_float2(scale, scale), make_float2(st.y, st.w)), prob);
                            };
                            // query ic + e sees key j from e = rel on
                            auto seen = [&](int e) { return (e < rel ? 0u : 0xFFFFu) | (e + 1 < rel ? 0u : 0xFFFF0000u); };
                            if (kTwoTerms) {  // of 16 columns, the second term's 8 after the first's
                                uint32_t rest_p[kPiece / 2], rest_d[kPiece / 2];
#pragma unroll
                                for (int e = 0; e < kPiece; e += 2) {
                                    float2 kept2, d;
                                    pair(e, kept2, d);
                                    const uint32_t mask = a.causal ? seen(e) : ~0u;
                                    s[e / 2] = pack2<T>(kept2.x, kept2.y), dp[e / 2] = pack2<T>(d.x, d.y);
                                    rest_p[e / 2] = rest2<T>(kept2, s[e / 2]) & mask, rest_d[e / 2] = rest2<T>(d, dp[e / 2]) & mask;
                                    s[e / 2] &= mask, dp[e / 2] &= mask;
                                }
#pragma unroll
                                for (int e = 0; e < kPiece / 2; e += 8) {
                                    const uint32_t to = mine + at + 2 * e;
                                    tmem_store(to, reinterpret_cast<const uint32_t(&)[8]>(s[e]));
                                    tmem_store(to + 8, reinterpret_cast<const uint32_t(&)[8]>(rest_p[e]));
                                    tmem_store(to + kCols, reinterpret_cast<const uint32_t(&)[8]>(dp[e]));
                                    tmem_store(to + kCols + 8, reinterpret_cast<const uint32_t(&)[8]>(rest_d[e]));
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < kPiece; e += 2) {
                                    float2 kept2, d;
                                    pair(e, kept2, d);
                                    s[e / 2] = pack2<T>(kept2.x, kept2.y), dp[e / 2] = pack2<T>(d.x, d.y);
                                }
                                if (a.causal && high > 0)
#pragma unroll
                                    for (int e = 0; e < kPiece; e += 2) s[e / 2] &= seen(e), dp[e / 2] &= seen(e);
                                const uint32_t to = mine + at / 32 * S::kPitch + at % 32 / 2;
                                tmem_store(to, reinterpret_cast<const uint32_t(&)[kPiece / 2]>(s));
                                tmem_store(to + kCols, reinterpret_cast<const uint32_t(&)[kPiece / 2]>(dp));
                            }
                        }
                        tmem_wait_store();
                    }
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(ready + 8 * chain);
                }
            };
            if (some) tiles(std::true_type{});
            else tiles(std::false_type{});
            use += w.tiles;

            // ---- the next item, and this one's result: chain 0's threads write dv, chain 1's dk
            const int32_t x = work.next_warp();
            const KeyItem next = x >= 0 ? key_item(p, x) : w;
            lost = fetch_lost(next);
            if (w.tiles) {
                barrier_wait(done, finished++ & 1u, &stalled);
                tmem_fence_after();
            }
            if (warp_j < a.len_k && chain < 2) {
                const Strides &st = chain ? a.dks : a.dvs;
                T *row = static_cast<T *>(chain ? a.dk : a.dv) + w.b * st.batch + j * st.len + w.head_kv * st.head;
                const float weight = chain ? a.scale : scale;
                constexpr int kParts = kDim / 32 / S::kShare;
#pragma unroll 1
                for (int c = 0; c < kParts; ++c) {
                    uint32_t o[32] = {};
                    const int col = 32 * (half * kParts + c);
                    if (w.tiles) {
                        tmem_load(o, (chain ? dk_at : dv_at) + lanes + col);
                        tmem_wait_load(o);
                    }
                    if (j < a.len_k) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float eight[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) eight[k] = j < w.keys ? __uint_as_float(o[e + k]) * weight : 0.0f;
                            if (col + e < a.dim) store<T, 8>(row + col + e, eight);
                        }
                    }
                }
            }
            // dv and dk have been read before the next item's first P is announced; and all leave together, also
            // when a wait of one of them ran out
            tmem_fence_before();
            if (!all_of<Team::kWorkers>(1, x >= 0)) break;
            w = next;
        }
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == Team::kMmaWarp) tmem_free<512>(tmem);
}

// ---- the table ---------------------------------------------------------------------

// dtable[n, head]: a block to each, its threads' sums over batch and query
// tiles added in a fixed order.
template <class T>
__global__ void __launch_bounds__(256) table_kernel(const __grid_constant__ BwdParams p)
{
    __shared__ float sums[8];
    const Attention &a = p.a;
    const int32_t n = blockIdx.y, head = blockIdx.x;
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
    size_t bias, sums, lost, floats;
};

BwdPlan bwd_plan(const Attention &a)
{
    BwdPlan f{};
    f.dim = a.dim <= 64 ? 64 : 128;
    f.pack = a.table ? 1 : packed_heads(a);
    f.units = a.batch * (a.heads / f.pack);
    const int32_t rows_per = kRows / f.pack;
    f.q_tiles = (a.len_q + rows_per - 1) / rows_per;
    f.len_pad = (a.len_q + kCols - 1) / kCols * kCols;
    const size_t heads = static_cast<size_t>(a.batch) * a.heads;
    f.bias = 2 * heads * f.len_pad;
    f.sums = f.bias + (a.table ? static_cast<size_t>(a.heads) * 2 * bias_reach(a.buckets) : 0);
    f.lost = f.sums + (a.dtable ? heads * f.q_tiles * a.buckets.total : 0);
    f.floats = f.lost + (a.table ? (heads * (f.len_pad / 32) + 3) / 4 : 0);
    return f;
}

template <class T, int kDim, bool kDrop, bool kBias, bool kTwoTerms>
cudaError_t launch_queries(const BwdParams &p, cudaStream_t s)
{
    const auto kernel = query_kernel<T, kDim, kDrop, kBias, kTwoTerms>;
    const size_t bytes = 1024 + QueryShape<kDim>::kTable + (kBias ? 2 * bias_reach(p.a.buckets) * (sizeof(float) + 1) : 0);
    static std::atomic<bool> done[16];
    const cudaError_t e = allow_shared(kernel, done);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(static_cast<int64_t>(p.units) * p.q_tiles), QueryShape<kDim>::Team::kThreads, bytes, s>>>(p);
    note_launch();
    return cudaGetLastError();
}

template <class T, int kDim, bool kDrop, bool kBias, bool kTwoTerms>
cudaError_t launch_keys(const BwdParams &p, cudaStream_t s)
{
    const auto kernel = key_kernel<T, kDim, kDrop, kBias, kTwoTerms>;
    const size_t bytes = 1024 + KeyShape<kDim>::kBytes;
    static std::atomic<bool> done[16];
    const cudaError_t e = allow_shared(kernel, done);
    if (e != cudaSuccess) return e;
    const int64_t blocks = static_cast<int64_t>(p.a.batch) * p.a.heads_kv * ((p.a.len_k + kRows - 1) / kRows);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    kernel<<<static_cast<unsigned>(blocks), KeyShape<kDim>::Team::kThreads, bytes, s>>>(p);
    note_launch();
    return cudaGetLastError();
}

template <class T, int kDim, bool kDrop, bool kBias, bool kTwoTerms>
cudaError_t launch_both(const BwdParams &p, bool queries, bool keys, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (queries) e = launch_queries<T, kDim, kDrop, kBias, kTwoTerms>(p, s);
    if (e == cudaSuccess && keys) e = launch_keys<T, kDim, kDrop, kBias, kTwoTerms>(p, s);
    return e;
}

template <class T, int kDim, bool kDrop, bool kBias>
cudaError_t launch_both(const BwdParams &p, bool queries, bool keys, cudaStream_t s)
{
    return two_terms(p.a) ? launch_both<T, kDim, kDrop, kBias, true>(p, queries, keys, s)
                          : launch_both<T, kDim, kDrop, kBias, false>(p, queries, keys, s);
}

template <class T, int kDim>
cudaError_t launch_both(const BwdParams &p, bool queries, bool keys, cudaStream_t s)
{
    const bool drop = p.a.mask.threshold != 0, bias = p.a.table != nullptr;
    if (drop)
        return bias ? launch_both<T, kDim, true, true>(p, queries, keys, s)
                    : launch_both<T, kDim, true, false>(p, queries, keys, s);
    return bias ? launch_both<T, kDim, false, true>(p, queries, keys, s)
                : launch_both<T, kDim, false, false>(p, queries, keys, s);
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
    p.pack = f.pack, p.pack_log = log2_of(f.pack), p.units = f.units, p.q_tiles = f.q_tiles, p.len_pad = f.len_pad;
    p.by_units = Divider(f.units), p.by_q_tiles = Divider(f.q_tiles), p.by_packs = Divider(a.heads / f.pack);
    p.by_group = Divider(a.group), p.by_key_units = Divider(a.batch * a.heads_kv), p.by_heads_kv = Divider(a.heads_kv);
    float *ws = static_cast<float *>(a.workspace);
    p.stats = reinterpret_cast<float2 *>(ws), p.bias = ws + f.bias, p.sums = ws + f.sums;
    p.lost = reinterpret_cast<uint8_t *>(ws + f.lost);
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
    // what is missing has no tile that is loaded, but a kernel prefetches its maps
    if (!has_q) p.q_cols = p.do_cols = p.k_cols;
    if (!has_k) p.k_cols = p.v_cols = p.q_cols;
    if (static_cast<int64_t>(f.units) * f.q_tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (e == cudaSuccess)
        e = f.dim == 64 ? launch_both<T, 64>(p, has_q, has_k, s) : launch_both<T, 128>(p, has_q, has_k, s);
    if (e == cudaSuccess && a.dtable && a.heads) {
        table_kernel<T><<<dim3(a.heads, a.buckets.total), 256, 0, s>>>(p);
        note_launch();
        e = cudaGetLastError();
    }
    return e;
}

template cudaError_t launch_attention_bwd<__half>(const Attention &, cudaStream_t);
template cudaError_t launch_attention_bwd<__nv_bfloat16>(const Attention &, cudaStream_t);

}  // namespace rngk
