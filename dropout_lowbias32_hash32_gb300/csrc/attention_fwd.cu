// attention_fwd.cu -- attention forward (include/rng.h, rng_attention_fwd) on
// the tensor cores.
//
// A block works on two units, each of 128 query rows with an O in TMEM.  A unit
// goes through tiles of 64 keys: S = Q K^T to TMEM, P = exp(S - max) written
// back over S in 16 bits, O += P V with P as the TMEM operand.  Two warpgroups
// take a unit's tiles in turn, a thread to a row, each with an S of its own: so
// four chains of product, exponential, product are under way, the tensor core
// works for three while the fourth computes, and four warps a scheduler hide each
// other's latencies.  One warp a unit issues its products, another the TMA loads; a
// stage of their ring holds a value tile and the key tile `kLead` after it.
//   kSplitKeys = false: the units are two tiles of queries that share the key
//     and value tiles (halving their traffic from L2);
//   kSplitKeys = true: one tile of queries, the units take every other key
//     tile and are joined at the end.  For one tile a head, where
//     the key axis may also be split over blocks, and is joined by join_kernel.
// The query heads of one key head are `pack` adjacent rows of a tile, so that
// they read its keys once.  A block that has finished takes over the work of one
// that has not started, so that its loads and first products run under the last
// of its previous work.
//
// A row's maximum passes from tile to tile through shared memory.  It is raised,
// and O rescaled, only when it has grown by more than 2^8: P then stays below
// 2^8, which 16 bits hold as well as 1.
//
// What bounds it, measured (bf16):
//   with dropout, the mask's hash: 10 of 17 instructions a pair (19 with a bias).
//     16 x 1024 positions, 16 heads of 64, 32 buckets, p = 0.1: 198 us, issue slots
//     72 % busy, ALU pipe 54 %, tensor core 15 %; without bias and dropout 97 us.
//   without it, the tensor core and what feeds it: 4099 causal positions, 32 heads
//     of 128 over 8 key heads: 106 us, 1.30 PFLOP/s of the visible pairs, tensor
//     core 60 %, exponentials 30 %.
//   for new tokens, HBM: 32 of them, 32 heads over 8 key heads of 128, 8192 cached
//     keys at most: 537 MB in 96 us, 5.6 TB/s, of which 5 us are join_kernel.
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace rngk {
namespace {

constexpr int kRows = 128, kKeys = 64;  // a unit's tile
// 2 x 2 warpgroups for the units, then a TMA warp, an MMA warp a unit, one that only fills the warpgroup
constexpr int kThreads = 640;
constexpr uint32_t kTmaWarp = 16, kMmaWarp = 17;
// registers: 640 threads start with 96 each; 4 x 104 + 64 = 5 x 96
constexpr int kUnitRegisters = 104, kOtherRegisters = 64;
constexpr uint32_t kRowsBox = 16384, kKeysBox = 8192;  // bytes of 128 and of 64 rows of 64 elements
constexpr float kLog2e = 1.4426950408889634f;

struct FwdParams {
    CUtensorMap q, k, v;
    Attention a;
    int32_t pack, pack_log, units, q_tiles, splits, split_tiles;
    Divider by_splits, by_units, by_q_tiles, by_packs, by_group;
    float *part;  // [splits][rows][dim padded + 2]: O, max, sum
};

template <int kDim, bool kSplitKeys>
struct Shape {
    static constexpr int kBoxes = kDim / 64;
    static constexpr int kQTiles = kSplitKeys ? 1 : 2;
    static constexpr int kLead = kSplitKeys ? 4 : 2;  // tiles whose S there is room for
    static constexpr int kStages = kDim == 64 ? 8 : 4;
    static constexpr uint32_t kRowsBytes = kBoxes * kRowsBox, kTileBytes = kBoxes * kKeysBox, kStageBytes = 2 * kTileBytes;
    static constexpr uint32_t kRing = kQTiles * kRowsBytes;                               // where the ring begins
    static constexpr uint32_t kHand = kRing + kStages * kStageBytes;                      // unit 1's O for unit 0, 64 columns at a time
    static constexpr uint32_t kTable = kHand + (kSplitKeys ? 64 * kRows * 4 : 0);  // a bias table a unit
};

// One item of work: a pack of heads of a batch entry, its query tiles, a range
// of key tiles.
struct Item {
    int32_t b, pack, head0, head_kv, i0, keys, pos0, split, tile0, count[2], tiles;
};

template <bool kSplitKeys>
__device__ __forceinline__ Item item_at(const FwdParams &p, uint32_t x)
{
    const Attention &a = p.a;
    Item w;
    int32_t rest, unit, q_tile;
    p.by_splits.divide(x, rest, w.split);
    if (a.causal) {  // the longest first
        p.by_units.divide(rest, q_tile, unit);
        q_tile = p.q_tiles - 1 - q_tile;
    } else {
        p.by_q_tiles.divide(rest, unit, q_tile);
    }
    const int32_t rows_per = kRows >> p.pack_log;  // positions of a tile
    p.by_packs.divide(unit, w.b, w.pack);
    w.head0 = w.pack << p.pack_log, w.head_kv = p.by_group.quotient(w.head0);
    w.i0 = q_tile * (kSplitKeys ? 1 : 2) * rows_per;
    w.keys = uniform(keys_of(a, w.b)), w.pos0 = first_position(a, w.keys);
    w.tile0 = w.split * p.split_tiles;
#pragma unroll
    for (int s = 0; s < 2; ++s) {  // key tiles of each unit (the item's, when the units share them out)
        const int32_t last = min(w.i0 + (kSplitKeys ? 1 : s + 1) * rows_per, a.len_q) - 1;  // the unit's last query
        int32_t end = a.causal ? min(w.keys, w.pos0 + last + 1) : w.keys;
        if (!kSplitKeys && w.i0 + s * rows_per >= a.len_q) end = 0;
        w.count[s] = max(0, min((end + kKeys - 1) / kKeys - w.tile0, p.split_tiles));
    }
    w.tiles = max(w.count[0], w.count[1]);
    return w;
}

template <class T, int kDim, bool kSplitKeys, bool kDrop, bool kBias, bool kTwoTerms>
__global__ void __launch_bounds__(kThreads, 1) attention_fwd_kernel(const __grid_constant__ FwdParams p)
{
    using S = Shape<kDim, kSplitKeys>;
    extern __shared__ uint8_t dynamic[];
    __shared__ alignas(16) uint4 response;
    __shared__ alignas(8) uint64_t bars[2 * S::kStages + 37];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t stalled;
    __shared__ float tops[2][2][kRows];                          // [unit][warpgroup][row], of its last tile
    __shared__ float last_tops[2][2][2][kRows], sums[2][2][2][kRows];  // [item's parity][unit][warpgroup][row]
    const Attention &a = p.a;
    const uint32_t warp = uniform(threadIdx.x / 32u), lane = threadIdx.x % 32u;
    uint8_t *smem = dynamic + ((1024u - (smem_address(dynamic) & 1023u)) & 1023u);
    const uint32_t base = smem_address(smem);

    // scored, ready: [unit][warpgroup]; passed: [unit][warpgroup][quarter]
    const uint32_t full = smem_address(bars), empty = full + 8 * S::kStages, scored = empty + 8 * S::kStages,
                   ready = scored + 32, passed = ready + 32, added = passed + 128, done = added + 16, q_full = done + 16, q_empty = q_full + 8,
                   tail = q_empty + 8, answered = tail + 8, heard = answered + 8, drained = heard + 8;
    if (threadIdx.x == 0) {
        prefetch_map(&p.q), prefetch_map(&p.k), prefetch_map(&p.v);
        stalled = 0;
        for (int s = 0; s < S::kStages; ++s) barrier_init(full + 8 * s, 1), barrier_init(empty + 8 * s, 2);
        for (int s = 0; s < 4; ++s) barrier_init(scored + 8 * s, 1), barrier_init(ready + 8 * s, 4);
        for (int s = 0; s < 16; ++s) barrier_init(passed + 8 * s, 1);
        for (int s = 0; s < 2; ++s) barrier_init(added + 8 * s, 1), barrier_init(done + 8 * s, 1);
        barrier_init(q_full, 1), barrier_init(q_empty, 2), barrier_init(tail, 1);
        barrier_init(answered, 1), barrier_init(heard, 18);
        for (int s = 0; s < 2; ++s) barrier_init(drained + 8 * s, 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc<512>(smem_address(&tmem_base));
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base;

    WorkQueue work{smem_address(&response), answered, heard, &stalled};

    if (warp >= kTmaWarp) {
        give_registers<kOtherRegisters>();
        if (warp == kTmaWarp) {
            // ---- TMA: the queries, then K_0 .. K_{lead-1} and alternately V_n, K_{n+lead}
            uint32_t use = 0, loaded = 0, tails = 0;
            bool fine = true;
            for (int32_t x = blockIdx.x; x >= 0 && fine; x = fine ? work.ask_warp() : -1) {
                const Item w = item_at<kSplitKeys>(p, x);
                if (w.tiles) {
                    if (loaded) fine = barrier_wait(q_empty, (loaded - 1) & 1u, &stalled);
                    if (!fine) break;
                    ++loaded;
                    if (elect_one()) {
                        barrier_expect(q_full, S::kQTiles * S::kRowsBytes);
                        for (int t = 0; t < S::kQTiles; ++t)
                            for (int c = 0; c < S::kBoxes; ++c)
                                tma_load_5d(base + t * S::kRowsBytes + c * kRowsBox, &p.q, q_full, c * 64, 0,
                                            w.i0 + t * (kRows >> p.pack_log), w.pack, w.b);
                    }
                }
#pragma unroll 1
                for (int32_t n = -S::kLead; n < w.tiles; ++n) {
                    const bool has_v = n >= 0, has_k = n + S::kLead < w.tiles;
                    if (!has_v && !has_k) continue;
                    const uint32_t stage = use % S::kStages, dst = base + S::kRing + stage * S::kStageBytes, bar = full + 8 * stage;
                    fine = barrier_wait(empty + 8 * stage, (use / S::kStages & 1u) ^ 1u, &stalled);
                    if (!fine) break;
                    ++use;
                    // values past n(b) that the array holds: whatever they are, P's zeros must meet zeros (the last
                    // tile's, which has no keys beside it)
                    const bool past = has_v && (w.tile0 + n + 1) * kKeys > w.keys && w.keys < a.len_k;
                    const uint32_t on = past ? tail : bar;
                    if (elect_one()) {
                        barrier_expect(on, (has_v && has_k ? 2 : 1) * S::kTileBytes);
#pragma unroll
                        for (int c = 0; c < S::kBoxes; ++c) {
                            if (has_v) tma_load_5d(dst + c * kKeysBox, &p.v, on, c * 64, 0, (w.tile0 + n) * kKeys, w.head_kv, w.b);
                            if (has_k)
                                tma_load_5d(dst + S::kTileBytes + c * kKeysBox, &p.k, on, c * 64, 0, (w.tile0 + n + S::kLead) * kKeys, w.head_kv, w.b);
                        }
                    }
                    if (past) {
                        if (!barrier_wait(tail, tails++ & 1u, &stalled)) barrier_drain(tail, (tails - 1) & 1u);
                        uint8_t *rows = smem + S::kRing + stage * S::kStageBytes;
                        for (int c = 0; c < S::kBoxes; ++c)
#pragma unroll 1
                            for (uint32_t o = (w.keys - (w.tile0 + n) * kKeys) * 128u + lane * 16u; o < kKeysBox; o += 512u)
                                *reinterpret_cast<uint4 *>(rows + c * kKeysBox + o) = make_uint4(0, 0, 0, 0);
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
        } else if (warp < kMmaWarp + 2) {
            // ---- MMA, a warp to a unit.  Both go through every stage, whether or not it holds something for their unit,
            // so that neither falls a whole phase behind.
            constexpr uint32_t kScores = mma_shape<T>(kKeys, false), kOut = mma_shape<T>(kDim, true);
            const uint32_t unit = warp - kMmaWarp, at = tmem + unit * 256;
            const uint64_t qd = row_major_tile(base + (kSplitKeys ? 0 : unit) * S::kRowsBytes);
            const uint64_t ring_v = column_major_tile(base + S::kRing, S::kBoxes > 1 ? kKeysBox : 1024);
            const uint64_t ring_k = row_major_tile(base + S::kRing + S::kTileBytes);
            uint32_t use = 0, given = 0, loaded = 0;  // given: bit g, the parity of warpgroup g's next P
            bool fine = true;
            for (int32_t x = blockIdx.x; x >= 0; x = fine ? work.next_warp() : -1) {
                const Item w = item_at<kSplitKeys>(p, x);
                if (!w.tiles) continue;
                const int32_t count = kSplitKeys ? w.tiles : unit ? w.count[1] : w.count[0];
                const uint32_t lead = min(w.tiles, S::kLead);
                fine = barrier_wait(q_full, loaded++ & 1u, &stalled);
                tmem_fence_after();
                bool scored_any = false;
#pragma unroll 1
                for (int32_t n = -S::kLead; n < w.tiles && fine; ++n) {
                    const int32_t next = n + S::kLead;
                    if (n < 0 && next >= w.tiles) continue;
                    const uint32_t u = use + (next < static_cast<int32_t>(lead) ? next : n + lead), stage = u % S::kStages;
                    const uint32_t group = (kSplitKeys ? next >> 1 : n) & 1u;  // tile n's and tile n + lead's
                    const bool mine = !kSplitKeys || (n & 1) == static_cast<int32_t>(unit), v_mine = mine && n >= 0 && n < count,
                               k_mine = mine && next < count;
                    fine = barrier_wait(full + 8 * stage, u / S::kStages & 1u, &stalled);
                    if (v_mine) {  // O += P V
                        fine = fine && barrier_wait(ready + 8 * (2 * unit + group), given >> group & 1u, &stalled);
                        given ^= 1u << group;
                    }
                    if (!fine) break;
                    tmem_fence_after();
                    if (elect_one()) {
                        if (v_mine) {
                            const uint64_t vd = ring_v + stage * (S::kStageBytes / 16);
#pragma unroll
                            for (int i = 0; i < kKeys / 16; ++i)
                                mma_step_tmem(at + 2 * kKeys, at + group * kKeys + i * 8, vd + i * (2048 / 16), kOut,
                                              n >= (kSplitKeys ? 2 : 1) || i > 0);
                            if (kTwoTerms)
#pragma unroll
                                for (int i = 0; i < kKeys / 16; ++i)
                                    mma_step_tmem(at + 2 * kKeys, at + group * kKeys + kKeys / 2 + i * 8, vd + i * (2048 / 16), kOut, true);
                            if (next >= count) mma_commit(added + 8 * unit);
                            if (n + (kSplitKeys ? 2 : 1) >= count) mma_commit(done + 8 * unit);
                        }
                        if (k_mine) {  // S = Q K^T
                            const uint64_t kd = ring_k + stage * (S::kStageBytes / 16);
#pragma unroll
                            for (int i = 0; i < kDim / 16; ++i)
                                mma_step(at + group * kKeys, qd + row_step(i, kRowsBox), kd + row_step(i, kKeysBox), kScores, i > 0);
                            mma_commit(scored + 8 * (2 * unit + group));
                        }
                        if (v_mine || k_mine) mma_commit(empty + 8 * stage);
                        else barrier_arrive(empty + 8 * stage);
                        if (k_mine && next + (kSplitKeys ? 2 : 1) >= count) mma_commit(q_empty);
                    }
                    scored_any = scored_any || k_mine;
                }
                if (!scored_any && elect_one()) barrier_arrive(q_empty);
                use += w.tiles + lead;
            }
            if (stalled && elect_one()) mma_commit(drained + 8 * unit), barrier_drain(drained + 8 * unit, 0);
        }
    } else {
        take_registers<kUnitRegisters>();
        // ---- the units' rows
        constexpr int kTogether = kSplitKeys ? 512 : 256;  // threads that work on an item's rows
        const int unit = warp / 8, group = warp / 4 % 2;
        const int32_t r = (warp % 4) * 32 + lane;
        const uint32_t lanes = (warp % 4) * 32u << 16, chain = 2 * unit + group;
        const uint32_t mine = tmem + unit * 256 + lanes + group * kKeys;              // the thread's scores, then its P
        const uint32_t out = tmem + unit * 256 + lanes + 2 * kKeys;
        const uint32_t pass = passed + 8 * (4 * chain + warp % 4), take = passed + 8 * (4 * (chain ^ 1) + warp % 4);
        const int32_t row0 = (kSplitKeys ? 0 : unit * kRows);
        // scores are held before or, with a bias, after their scaling; base two is for the exponential
        const float to_base2 = kBias ? kLog2e : a.scale * kLog2e;
        const int32_t reach = kBias ? bias_reach(a.buckets) : 0;
        float *table = reinterpret_cast<float *>(smem + S::kTable) + unit * 2 * reach;
        int32_t table_head = -1;
        uint32_t turn = 0, turns_of_other = 0, taken = 0, additions = 0, finished = 0, item = 0;
        Item w = item_at<kSplitKeys>(p, blockIdx.x);
        for (;; ++item) {
            const int32_t warp_i = w.i0 + ((row0 + (warp % 4) * 32) >> p.pack_log);  // the warp's first query
            const int32_t i = w.i0 + ((row0 + r) >> p.pack_log), head = w.head0 + (r & (p.pack - 1)), pos = w.pos0 + i;
            const bool valid = i < a.len_q, any = warp_i < a.len_q;
            const int64_t index = (static_cast<int64_t>(w.b) * a.heads + head) * a.len_q + i;
            const uint32_t counter = a.first + static_cast<uint32_t>(index) * static_cast<uint32_t>(a.len_k);
            const int32_t visible = a.causal ? min(w.keys, pos + 1) : w.keys;
            const int32_t warp_visible = a.causal ? min(w.keys, w.pos0 + warp_i + 1) : w.keys;  // the least of the warp's
            if (kBias && w.head0 != table_head) {  // the bias by relative position (pack is 1)
                table_head = w.head0;
                sync_threads<256>(2 + unit);
                for (int32_t t = threadIdx.x % 256u; t < 2 * reach; t += 256)
                    table[t] = a.table ? to_f32(static_cast<const T *>(a.table)[bucket_of(a.buckets, t - reach) * a.heads + w.head0]) : 0.0f;
                sync_threads<256>(2 + unit);
            }
            float top = -INFINITY, sum = 0.0f;
            // the unit's tiles; this warpgroup's are group, group + 2, ...
            const int32_t count = kSplitKeys ? (w.tiles + 1 - unit) / 2 : unit ? w.count[1] : w.count[0];
#pragma unroll 1
            for (int32_t j = group; j < count; j += 2, ++turn) {
                const int32_t j0 = (w.tile0 + (kSplitKeys ? 2 * j + unit : j)) * kKeys;
                barrier_wait(scored + 8 * chain, turn & 1u, &stalled);
                tmem_fence_after();
                if (any) {
                    uint32_t s[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_load(s[c], mine + 32 * c);
                    tmem_wait_load(s[0], s[1]);
                    if (kBias) {
                        // relative positions of the warp's pairs: beyond the last bucket's start on one side, or by the table
                        const int32_t low = j0 - (w.pos0 + warp_i + 31), high = j0 + kKeys - 1 - (w.pos0 + warp_i);
                        const float2 scale = make_float2(a.scale, a.scale);
                        if (high <= -a.buckets.max_distance || low >= a.buckets.max_distance) {
                            const float v = table[high < 0 ? 0 : 2 * reach - 1];
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 f = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), scale, make_float2(v, v));
                                    s[c][e] = __float_as_uint(f.x), s[c][e + 1] = __float_as_uint(f.y);
                                }
                        } else {
                            const float *t = table + (j0 - pos + reach);
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 f = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), scale,
                                                          make_float2(t[32 * c + e], t[32 * c + e + 1]));
                                    s[c][e] = __float_as_uint(f.x), s[c][e + 1] = __float_as_uint(f.y);
                                }
                        }
                    }
                    if (j0 + kKeys > warp_visible) {
                        const int32_t seen = visible - j0;
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * c + e >= seen) s[c][e] = __float_as_uint(-INFINITY);
                    }
                    float most[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t(&q)[16] = *reinterpret_cast<const uint32_t(*)[16]>(&s[c / 2][c % 2 * 16]);
                        most[c] = __uint_as_float(q[0]);
#pragma unroll
                        for (int e = 1; e < 15; e += 2) most[c] = max3(most[c], __uint_as_float(q[e]), __uint_as_float(q[e + 1]));
                        most[c] = fmaxf(most[c], __uint_as_float(q[15]));
                    }
                    const float tile_top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
                    // the maximum after the unit's previous tile, to which this warpgroup's sum is brought
                    if (j > 0) {
                        barrier_wait(take, taken++ & 1u, &stalled);
                        const float given = tops[unit][group ^ 1][r];
                        if (given > top) {
                            sum *= exp2_approx((top - given) * to_base2);
                            top = given;
                        }
                    }
                    // a new one, and O and the sum brought to it: at the first finite score, or 2^8 above the old one
                    const bool raise = tile_top > top && (top == -INFINITY || (tile_top - top) * to_base2 > 8.0f);
                    if (__any_sync(0xFFFFFFFFu, raise)) {
                        const float fade = raise ? exp2_approx((top - tile_top) * to_base2) : 1.0f;
                        sum *= fade;
                        if (raise) top = tile_top;
                        if (j > 0) {
                            // O up to the previous tile: what was issued after its product tells (the one before
                            // that was added before this S was made)
                            if (j + 1 < count) barrier_wait(scored + 8 * (chain ^ 1), (turns_of_other + (j + 1) / 2) & 1u, &stalled);
                            else barrier_wait(added + 8 * unit, (additions + j - 1 - max(count - 2, 0)) & 1u, &stalled);
                            tmem_fence_after();
#pragma unroll 1
                            for (int c = 0; c < kDim / 16; ++c) {
                                uint32_t o[16];
                                tmem_load(o, out + 16 * c);
                                tmem_wait_load(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fade);
                                tmem_store(out + 16 * c, o);
                            }
                        }
                    }
                    tops[unit][group][r] = top;
                    __syncwarp();
                    if (lane == 0) barrier_arrive(pass);
                    // exp2((s - top) to_base2): as one multiply-add, or, where a bias may be the type's
                    // lowest value, with the difference taken first
                    const float from = top == -INFINITY ? 0.0f : -top, shift = from * to_base2;
                    const float2 from2 = make_float2(from, from), shift2 = make_float2(shift, shift);
                    const float2 base2 = make_float2(to_base2, to_base2);
                    auto exponentials = [&](int c, uint32_t e) {
                        const float2 v = make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                        const float2 f = kBias ? mul2(add2(v, from2), base2) : fma2(v, base2, shift2);
                        return make_float2(exp2_approx(f.x), exp2_approx(f.y));
                    };
                    float2 total = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t q[16], rest[8];  // (which rounding left, 16 columns at a time)
                        for_pairs32<kDrop>(a.mask, counter + j0 + 32 * c, [&](uint32_t e, float2 k) {
                            float2 x = exponentials(c, e);
                            total = add2(total, x);
                            if (kDrop) x = mul2(x, k);
                            q[e / 2] = pack2<T>(x.x, x.y);
                            if constexpr (kTwoTerms) {
                                rest[e / 2 % 8] = rest2<T>(x, q[e / 2]);
                                if (e % 16 == 14) tmem_store(mine + kKeys / 2 + 16 * c + e / 16 * 8, rest);  // beside P
                            }
                        });
                        tmem_store(mine + 16 * c, q);
                    }
                    sum += total.x + total.y;
                    tmem_wait_store();
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(ready + 8 * chain);
            }
            // the other warpgroup's maxima that this one had no tile for
            if (any) taken += group ? 0 : (count > 0 ? count / 2 - (count - 1) / 2 : 0);
            if (any && group) taken += (count + 1) / 2 - count / 2;

            // ---- the next item, and this one's result
            const int32_t x = work.next_warp();
            const Item next = x >= 0 ? item_at<kSplitKeys>(p, x) : w;
            const bool two = kSplitKeys && w.tiles > 1;
            if (count) {
                barrier_wait(done + 8 * unit, finished++ & 1u, &stalled);
                tmem_fence_after();
            }
            additions += min(count, 2);
            turns_of_other += group ? (count + 1) / 2 : count / 2;
            float(&all_tops)[2][2][kRows] = last_tops[item & 1u], (&all_sums)[2][2][kRows] = sums[item & 1u];
            all_tops[unit][group][r] = top, all_sums[unit][group][r] = sum;
            sync_threads<kTogether>(kSplitKeys ? 1 : 2 + unit);
            // the warpgroups' maxima only grow, so O is relative to the larger
            auto whole_unit = [&](int u, float &most, float &total) {
                const float t0 = all_tops[u][0][r], t1 = all_tops[u][1][r];
                most = fmaxf(t0, t1);
                // (without a maximum, the sum is 0, or NaN where the scores are)
                total = all_sums[u][0][r] * (t0 == -INFINITY ? 1.0f : exp2_approx((t0 - most) * to_base2)) +
                        all_sums[u][1][r] * (t1 == -INFINITY ? 1.0f : exp2_approx((t1 - most) * to_base2));
            };
            float weight = 1.0f, other = 0.0f;
            whole_unit(kSplitKeys ? 0 : unit, top, sum);
            if (two) {
                float top1, sum1;
                whole_unit(1, top1, sum1);
                const float most = fmaxf(top, top1);
                weight = top == -INFINITY ? 0.0f : exp2_approx((top - most) * to_base2);
                other = top1 == -INFINITY ? 0.0f : exp2_approx((top1 - most) * to_base2);
                sum = sum * weight + sum1 * other;
                top = most;
            }
            const float to_natural = kBias ? 1.0f : a.scale;
            const bool whole = p.splits == 1, mine_to_write = !kSplitKeys || unit == 0;
            float *part = p.part + (static_cast<int64_t>(w.split) * a.batch * a.heads * a.len_q + index) * (kDim + 2);
            const float scale = !whole ? 1.0f : sum == 0.0f ? 0.0f : a.mask.scale / sum;
            T *o_row = static_cast<T *>(a.out) + w.b * a.os.batch + i * a.os.len + head * a.os.head;
            float *hand = reinterpret_cast<float *>(smem + S::kHand) + group * 32 * kRows + r;
#pragma unroll 1
            for (int c = 0; c < kDim / 64; ++c) {
                uint32_t o[32] = {};
                const int col = group * (kDim / 2) + 32 * c;
                if (count && any) {
                    tmem_load(o, out + col);
                    tmem_wait_load(o);
                }
                if (two) {  // unit 1 hands its part to unit 0
                    if (c) sync_threads<512>(1);
                    if (unit == 1 && any) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) hand[e * kRows] = __uint_as_float(o[e]);
                    }
                    sync_threads<512>(1);
                }
                if (valid && mine_to_write) {
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        v[e] = __uint_as_float(o[e]);
                        if (two) v[e] = v[e] * weight + hand[e * kRows] * other;
                        if (sum == 0.0f) v[e] = 0.0f;  // nothing seen
                        v[e] *= scale;
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            const float(&eight)[8] = *reinterpret_cast<const float(*)[8]>(&v[e]);
                            if (col + e < a.dim) store<T, 8>(o_row + col + e, eight);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) *reinterpret_cast<float2 *>(part + col + e) = make_float2(v[e], v[e + 1]);
                    }
                }
            }
            if (valid && mine_to_write && group == 0) {
                if (!whole)
                    part[kDim] = top * to_natural, part[kDim + 1] = sum;
                else if (a.lse)
                    a.lse[index] = sum == 0.0f ? -INFINITY : top * to_natural + logf(sum);
            }
            // Both warpgroups have read O before the next item's first P is announced; and they leave together, also
            // when a wait of one of them ran out.
            tmem_fence_before();
            if (!all_of<kTogether>(kSplitKeys ? 1 : 2 + unit, x >= 0)) break;
            w = next;
        }
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) tmem_free<512>(tmem);
}

// Joins the key axis's splits: a warp to a row, the loads of four splits at
// once (one that saw no key has the maximum -inf and zeros).
template <class T, int kDim>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ FwdParams p)
{
    const Attention &a = p.a;
    const int64_t rows = static_cast<int64_t>(a.batch) * a.heads * a.len_q;
    const int64_t index = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.y;
    if (index >= rows) return;
    const uint32_t lane = threadIdx.x;
    constexpr int kEach = kDim / 32, kAtOnce = 4;
    float top = -INFINITY, sum = 0.0f, o[kEach] = {};
    for (int32_t s = 0; s < p.splits; s += kAtOnce) {
        float2 stats[kAtOnce], part[kAtOnce][kEach / 2];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const float2 *at = reinterpret_cast<const float2 *>(p.part + (min(s + u, p.splits - 1) * rows + index) * (kDim + 2));
            stats[u] = at[kDim / 2];
#pragma unroll
            for (int k = 0; k < kEach / 2; ++k) part[u][k] = at[lane * (kEach / 2) + k];
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (s + u >= p.splits || stats[u].y == 0.0f) continue;
            const float next = fmaxf(top, stats[u].x), fade = exp2_approx((top - next) * kLog2e);
            const float weight = exp2_approx((stats[u].x - next) * kLog2e);
            sum = sum * fade + stats[u].y * weight;
            top = next;
#pragma unroll
            for (int k = 0; k < kEach; ++k) o[k] = o[k] * fade + (k % 2 ? part[u][k / 2].y : part[u][k / 2].x) * weight;
        }
    }
    const int64_t i = index % a.len_q, h = index / a.len_q % a.heads, b = index / a.len_q / a.heads;
    const float scale = sum == 0.0f ? 0.0f : a.mask.scale / sum;
    T *row = static_cast<T *>(a.out) + b * a.os.batch + i * a.os.len + h * a.os.head;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (lane * kEach + k < a.dim) row[lane * kEach + k] = from_f32<T>(o[k] * scale);
    if (a.lse && lane == 0) a.lse[index] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

// How a call is cut.
struct FwdPlan {
    int32_t dim, pack, units, q_tiles, splits, split_tiles;
    bool split_keys;
};

FwdPlan fwd_plan(const Attention &a)
{
    FwdPlan f;
    f.dim = a.dim <= 64 ? 64 : 128;
    f.pack = packed_heads(a);
    f.units = a.batch * (a.heads / f.pack);
    const int32_t rows_per = kRows / f.pack, tiles = (a.len_q + rows_per - 1) / rows_per;
    const int32_t key_tiles = (a.len_k + kKeys - 1) / kKeys;
    f.split_keys = tiles == 1;
    f.q_tiles = f.split_keys ? tiles : (tiles + 1) / 2;
    f.splits = 1, f.split_tiles = key_tiles < 1 ? 1 : key_tiles;
    if (f.split_keys && key_tiles > 8) {
        // about four blocks to an SM, of eight key tiles or more (the second launch that joins them costs as much as
        // some six tiles)
        const int64_t blocks = static_cast<int64_t>(f.units) * f.q_tiles, want = (4ll * sm_count() + blocks - 1) / blocks;
        const int64_t most = (key_tiles + 7) / 8;
        const int64_t splits = want < most ? want : most;
        f.split_tiles = static_cast<int32_t>((key_tiles + splits - 1) / splits);
        f.splits = (key_tiles + f.split_tiles - 1) / f.split_tiles;
    }
    return f;
}

template <class T, int kDim, bool kSplitKeys, bool kDrop, bool kBias, bool kTwoTerms>
cudaError_t launch(const FwdParams &p, cudaStream_t s)
{
    using S = Shape<kDim, kSplitKeys>;
    const auto kernel = attention_fwd_kernel<T, kDim, kSplitKeys, kDrop, kBias, kTwoTerms>;
    const size_t bytes = 1024 + S::kTable + (kBias ? 4 * bias_reach(p.a.buckets) * sizeof(float) : 0);
    static std::atomic<bool> done[16];
    const cudaError_t e = allow_shared(kernel, done);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(static_cast<int64_t>(p.units) * p.q_tiles * p.splits), kThreads, bytes, s>>>(p);
    note_launch();
    if (p.splits > 1) {
        const int64_t rows = static_cast<int64_t>(p.a.batch) * p.a.heads * p.a.len_q;
        join_kernel<T, kDim><<<static_cast<unsigned>((rows + 3) / 4), dim3(32, 4), 0, s>>>(p);
        note_launch();
    }
    return cudaGetLastError();
}

template <class T, int kDim, bool kSplitKeys, bool kTwoTerms>
cudaError_t launch(const FwdParams &p, cudaStream_t s)
{
    const bool drop = p.a.mask.threshold != 0, bias = has_bias(p.a);
    if (drop)
        return bias ? launch<T, kDim, kSplitKeys, true, true, kTwoTerms>(p, s)
                    : launch<T, kDim, kSplitKeys, true, false, kTwoTerms>(p, s);
    return bias ? launch<T, kDim, kSplitKeys, false, true, kTwoTerms>(p, s)
                : launch<T, kDim, kSplitKeys, false, false, kTwoTerms>(p, s);
}

template <class T, int kDim>
cudaError_t launch(const FwdParams &p, bool split_keys, cudaStream_t s)
{
    if (two_terms(p.a)) return split_keys ? launch<T, kDim, true, true>(p, s) : launch<T, kDim, false, true>(p, s);
    return split_keys ? launch<T, kDim, true, false>(p, s) : launch<T, kDim, false, false>(p, s);
}

}  // namespace

cudaError_t stalled_waits_fwd(uint64_t *count)
{
    return cudaMemcpyFromSymbol(count, g_stalled_waits, sizeof(uint64_t));
}

size_t attention_fwd_workspace(const Attention &a)
{
    if (a.batch == 0 || a.len_q == 0 || a.heads == 0) return 0;
    const FwdPlan f = fwd_plan(a);
    if (f.splits == 1) return 0;
    return static_cast<size_t>(f.splits) * a.batch * a.heads * a.len_q * (f.dim + 2) * sizeof(float);
}

template <class T>
cudaError_t launch_attention_fwd(const Attention &a, cudaStream_t s)
{
    const FwdPlan f = fwd_plan(a);
    FwdParams p;
    p.a = a;
    p.pack = f.pack, p.units = f.units, p.q_tiles = f.q_tiles, p.splits = f.splits, p.split_tiles = f.split_tiles;
    p.pack_log = log2_of(f.pack);
    p.by_splits = Divider(f.splits), p.by_units = Divider(f.units), p.by_q_tiles = Divider(f.q_tiles);
    p.by_packs = Divider(a.heads / f.pack), p.by_group = Divider(a.group);
    p.part = static_cast<float *>(a.workspace);
    if (static_cast<int64_t>(f.units) * f.q_tiles * f.splits > 0x7FFFFFFF) return cudaErrorInvalidValue;
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    cudaError_t e = make_heads_map(&p.q, bf16, a.q, a.qs, a.batch, a.len_q, a.heads, a.dim, f.pack, kRows);
    if (a.len_k > 0) {
        if (e == cudaSuccess) e = make_heads_map(&p.k, bf16, a.k, a.ks, a.batch, a.len_k, a.heads_kv, a.dim, 1, kKeys);
        if (e == cudaSuccess) e = make_heads_map(&p.v, bf16, a.v, a.vs, a.batch, a.len_k, a.heads_kv, a.dim, 1, kKeys);
    } else {
        p.k = p.v = p.q;  // not read
    }
    if (e != cudaSuccess) return e;
    return f.dim == 64 ? launch<T, 64>(p, f.split_keys, s) : launch<T, 128>(p, f.split_keys, s);
}

template cudaError_t launch_attention_fwd<__half>(const Attention &, cudaStream_t);
template cudaError_t launch_attention_fwd<__nv_bfloat16>(const Attention &, cudaStream_t);

}  // namespace rngk
