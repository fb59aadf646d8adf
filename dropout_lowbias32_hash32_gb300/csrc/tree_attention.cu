// tree_attention.cu -- attention of a tree of drafted tokens over a cache
// (include/rng.h, rng_tree_attention_fwd) on the tensor cores.
//
// The rows of a key head, its query heads' nodes, are packed into tiles of 128,
// so that its keys are read once; two units a block, each with a tile of rows, an S
// and an O in TMEM and a warpgroup, a row to a thread:
//   kTiles = 1 (at most 128 rows): the units take every other tile of 128 keys
//     and are joined at the end;
//   kTiles = 2: the units have two tiles of rows and share the key tiles.
// A unit's step is S = Q K^T, P = exp(S - max) written back over S in 16 bits, O +=
// P V; one warp issues both units' products in turn, so that one unit's
// exponentials run under the other's products.  One warp issues the TMA loads, one
// clears value rows that nobody may look at.
//
// The work is the list of all (batch entry, key head, rows) and their key tiles,
// cut evenly among the blocks by the lengths found on the device.  A block's first
// and last piece may be a part of one entry's keys; join_kernel puts parts together.
//
// A row's maximum is raised, and O rescaled, only when it has grown by more than
// 2^8: P then stays below 2^8, which 16 bits hold as well as 1.
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace rngk {
namespace {

constexpr int kRows = 128, kKeys = 128;  // a unit's tile
constexpr int kThreads = 384;            // a warpgroup a unit, and one of the TMA, MMA and clearing warps
constexpr uint32_t kTmaWarp = 8, kMmaWarp = 9, kClearWarp = 10;
// registers: 384 threads start with 168 each; 2 x 208 + 80 <= 3 x 168
constexpr int kUnitRegisters = 208, kOtherRegisters = 80;
constexpr uint32_t kBox = 16384;  // bytes of 128 rows of 64 elements
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxNodes = RNG_MAX_TREE_NODES;
constexpr int kTableValues = 1024;  // bias values of a pack of heads in shared memory
constexpr int kLeastPart = 2;       // key tiles of a part at least
constexpr int kOddBuffers = 8;

using Bits = unsigned __int128;
static_assert(kMaxNodes == 128, "a node's line is a 128-bit mask");

struct TreeParams {
    CUtensorMap q, k, v;
    TreeAttention t;
    // heads side by side in a tile, nodes of a tile, packs of heads, pairs (kTiles = 1: single ones) of tiles of a pack,
    // packs x pairs, rows of a part
    int32_t pack, nodes_per, packs, pairs, units, part_rows;
    float *part;  // [blocks][2][part_rows][dim padded + 2]: O, max, sum
    int4 *meta;   // [blocks][2]: batch entry, unit, first key tile, state
};

// A part's state.
constexpr int32_t kIsThere = 1, kIsPart = 2, kStarts = 4, kEnds = 8;

template <int kDim, int kTiles>
struct Shape {
    static constexpr int kBoxes = kDim / 64;
    static constexpr int kQBuffers = 3 - kTiles;
    static constexpr int kStages = kDim == 64 ? 8 : 4;
    static constexpr uint32_t kTileBytes = kBoxes * kBox;
    static constexpr uint32_t kRing = 2 * kTileBytes;                                     // after two tiles of queries
    static constexpr uint32_t kHand = kRing + kStages * kTileBytes;                       // unit 1's O for unit 0, 32 columns at a time
    static constexpr uint32_t kTable = kHand + (kTiles == 1 ? 32 * kRows * 4 : 0);        // bias values a unit
    static constexpr uint32_t kBuckets = kTable + 2 * kTableValues * 4;                   // bucket by distance
};

__device__ __forceinline__ int32_t cached_of(const Attention &a, int32_t b)
{
    const int32_t room = a.len_k - a.len_q;
    return a.key_lengths ? min(max(a.key_lengths[b], 0), room) : room;
}
__device__ __forceinline__ int32_t tiles_of(const Attention &a, int32_t b) { return (cached_of(a, b) + a.len_q + kKeys - 1) / kKeys; }

// A run of one unit's key tiles.
struct Piece {
    int32_t b, unit, tile0, tiles, all;  // all: of the unit
    int32_t cached, pack, head0, head_kv, node0;
    bool second;  // (kTiles = 2) whether the second tile has rows
};

// A block's pieces, one after the other.
struct Cursor {
    int64_t at, end, base;  // in the list of all key tiles; base: where the batch entry's begin
    int32_t b, tiles;       // its key tiles of one unit

    template <int kTiles>
    __device__ __forceinline__ bool next(const TreeParams &p, Piece &w)
    {
        if (at >= end) return false;
        const Attention &a = p.t.a;
        while (at >= base + static_cast<int64_t>(tiles) * p.units) {
            base += static_cast<int64_t>(tiles) * p.units;
            tiles = uniform(tiles_of(a, ++b));
        }
        const uint64_t local = at - base;
        w.b = b, w.all = tiles;
        w.unit = static_cast<int32_t>(local / static_cast<uint32_t>(tiles));
        w.tile0 = static_cast<int32_t>(local - static_cast<uint64_t>(w.unit) * tiles);
        const int64_t left = end - at;
        w.tiles = w.all - w.tile0 < left ? w.all - w.tile0 : static_cast<int32_t>(left);
        at += w.tiles;
        w.cached = uniform(cached_of(a, b));
        const int32_t pair = w.unit % p.pairs;
        w.pack = w.unit / p.pairs;
        w.head0 = w.pack * p.pack, w.head_kv = w.head0 / a.group;
        w.node0 = pair * kTiles * p.nodes_per;
        w.second = kTiles == 2 && w.node0 + p.nodes_per < a.len_q;
        return true;
    }
};

// Where the list is cut at x: at a unit's own beginning or end rather than less than kLeastPart tiles from it.
__device__ __forceinline__ int64_t snapped(int64_t x, int64_t base, int32_t tiles)
{
    const int32_t o = static_cast<int32_t>(static_cast<uint64_t>(x - base) % static_cast<uint32_t>(tiles));
    return o < kLeastPart ? x - o : tiles - o < kLeastPart ? x - o + tiles : x;
}

template <class T, int kDim, int kTiles, bool kBias>
__global__ void __launch_bounds__(kThreads, 1) tree_attention_kernel(const __grid_constant__ TreeParams p)
{
    using S = Shape<kDim, kTiles>;
    constexpr bool kTwoTerms = kTiles == 1;
    // f16 holds 2^15: P below 2^8 is lifted, so that long rows' small ones keep their bits
    constexpr float kLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;
    extern __shared__ uint8_t dynamic[];
    __shared__ alignas(8) uint64_t bars[3 * S::kStages + 12];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t stalled;
    __shared__ Cursor shared_cursor;
    __shared__ int64_t scan[kThreads / 32 + 1], cut_end;
    __shared__ Bits seen_by[2][kMaxNodes];      // [unit][node]: the nodes of its line, none for an absent one
    __shared__ int16_t depth_by[2][kMaxNodes];  // nodes before it
    __shared__ uint32_t odd[kOddBuffers][4];    // nodes with an infinity or NaN among their values
    __shared__ float tops[2][kRows], sums[2][kRows];
    const Attention &a = p.t.a;
    const uint32_t warp = uniform(threadIdx.x / 32u), lane = threadIdx.x % 32u;
    uint8_t *smem = dynamic + ((1024u - (smem_address(dynamic) & 1023u)) & 1023u);
    const uint32_t base = smem_address(smem);

    const uint32_t full = smem_address(bars), empty = full + 8 * S::kStages, tail = empty + 8 * S::kStages,
                   scored = tail + 8 * S::kStages, ready = scored + 16, done = ready + 16, q_full = done + 16,
                   q_empty = q_full + 16, drained = q_empty + 16;
    if (threadIdx.x == 0) {
        prefetch_map(&p.q), prefetch_map(&p.k), prefetch_map(&p.v);
        stalled = 0;
        for (int s = 0; s < S::kStages; ++s) barrier_init(full + 8 * s, 1), barrier_init(empty + 8 * s, 1), barrier_init(tail + 8 * s, 1);
        for (int s = 0; s < 2; ++s)
            barrier_init(scored + 8 * s, 1), barrier_init(ready + 8 * s, 4), barrier_init(done + 8 * s, 1),
                barrier_init(q_full + 8 * s, 1), barrier_init(q_empty + 8 * s, 1);
        barrier_init(drained, 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc<512>(smem_address(&tmem_base));
    if (kBias && a.table) {
        uint8_t *bucket = smem + S::kBuckets;
        for (int32_t d = threadIdx.x; d <= a.buckets.max_distance; d += kThreads) bucket[d] = static_cast<uint8_t>(bucket_of(a.buckets, -d));
    }

    // ---- the block's share of the list
    auto block_sum = [&](int64_t v, int64_t &before) {  // over the threads; before: over those before this one
        int64_t up_to = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, up_to, d);
            if (lane >= static_cast<uint32_t>(d)) up_to += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = up_to;
        __syncthreads();
        before = up_to - v;
        int64_t all = 0;
        for (uint32_t w = 0; w < kThreads / 32; ++w) {
            if (w == warp) before += all;
            all += scan[w];
        }
        return all;
    };
    {
        int64_t mine = 0, before;
        for (int32_t b = threadIdx.x; b < a.batch; b += kThreads) mine += tiles_of(a, b);
        const int64_t all = block_sum(mine, before) * p.units;
        const int64_t from = all * blockIdx.x / gridDim.x, to = all * (blockIdx.x + 1) / gridDim.x;
        if (threadIdx.x == 0) shared_cursor = Cursor{all, all, all, a.batch - 1, 1}, cut_end = all;
        int64_t so_far = 0;
        for (int32_t b0 = 0; b0 < a.batch; b0 += kThreads) {
            const int32_t b = b0 + static_cast<int32_t>(threadIdx.x), n = b < a.batch ? tiles_of(a, b) : 0;
            const int64_t part = block_sum(static_cast<int64_t>(n) * p.units, before), begin = so_far + before,
                          past = begin + static_cast<int64_t>(n) * p.units;
            if (from >= begin && from < past) shared_cursor = Cursor{snapped(from, begin, n), 0, begin, b, n};
            if (to >= begin && to < past) cut_end = snapped(to, begin, n);
            so_far += part;
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base;
    Cursor cursor = shared_cursor;
    cursor.end = cut_end;
    Piece w;

    if (warp >= kTmaWarp) {
        give_registers<kOtherRegisters>();
        if (warp == kTmaWarp) {
            // ---- TMA: a piece's queries, then its keys and values in the order in which the products take them
            uint32_t use = 0, piece = 0, on_tail = 0, tail_turns = 0;  // bit s: stage s's last tile, the parity of its next
            bool fine = true;
            while (fine && cursor.next<kTiles>(p, w)) {
                const uint32_t buffer = piece % S::kQBuffers, before = piece / S::kQBuffers;
                if (before) fine = barrier_wait(q_empty + 8 * buffer, (before - 1) & 1u, &stalled);
                if (!fine) break;
                ++piece;
                if (elect_one()) {
                    const uint32_t rows = p.pack * p.nodes_per * 128u;
                    barrier_expect(q_full + 8 * buffer, kTiles * S::kBoxes * rows);
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
#pragma unroll
                        for (int c = 0; c < S::kBoxes; ++c)
                            tma_load_5d(base + (kTiles == 2 ? t : buffer) * S::kTileBytes + c * kBox, &p.q, q_full + 8 * buffer, c * 64, 0,
                                        w.node0 + t * p.nodes_per, w.pack, w.b);
                }
                auto tile = [&](bool value, int32_t n) {
                    const uint32_t stage = use % S::kStages, dst = base + S::kRing + stage * S::kTileBytes;
                    fine = barrier_wait(empty + 8 * stage, (use / S::kStages & 1u) ^ 1u, &stalled);
                    if (!fine) return;
                    ++use;
                    // value rows from the tree on are looked through before the products see them
                    const bool looked_through = value && (w.tile0 + n + 1) * kKeys > w.cached;
                    const uint32_t bar = (looked_through ? tail : full) + 8 * stage;
                    on_tail = looked_through ? on_tail | 1u << stage : on_tail & ~(1u << stage);
                    tail_turns ^= looked_through ? 1u << stage : 0u;
                    if (elect_one()) {
                        barrier_expect(bar, S::kTileBytes);
#pragma unroll
                        for (int c = 0; c < S::kBoxes; ++c)
                            tma_load_5d(dst + c * kBox, value ? &p.v : &p.k, bar, c * 64, 0, (w.tile0 + n) * kKeys, w.head_kv, w.b);
                    }
                };
                constexpr int32_t kLead = kTiles == 1 ? 2 : 1;
                for (int32_t n = 0; n < kLead && n < w.tiles && fine; ++n) tile(false, n);
                for (int32_t n = 0; n < w.tiles && fine; ++n) {
                    tile(true, n);
                    if (fine && n + kLead < w.tiles) tile(false, n + kLead);
                }
            }
            if (stalled) {  // nothing may land after the block has ended
                for (uint32_t b = 0; b < S::kQBuffers; ++b)
                    if (piece > b) barrier_drain(q_full + 8 * b, ((piece - 1 - b) / S::kQBuffers) & 1u);
                for (uint32_t u = use > S::kStages ? use - S::kStages : 0; u < use; ++u) {
                    const uint32_t stage = u % S::kStages;
                    if (on_tail >> stage & 1u) barrier_drain(tail + 8 * stage, (tail_turns >> stage & 1u) ^ 1u);
                    else barrier_drain(full + 8 * stage, u / S::kStages & 1u);
                }
            }
        } else if (warp == kMmaWarp) {
            // ---- MMA
            constexpr uint32_t kScores = mma_shape<T>(kKeys, false), kOut = mma_shape<T>(kDim, true);
            const uint64_t ring_v = column_major_tile(base + S::kRing, S::kBoxes > 1 ? kBox : 1024);
            const uint64_t ring_k = row_major_tile(base + S::kRing), qd = row_major_tile(base);
            uint32_t use = 0, piece = 0, given = 0;  // given: bit u, the parity of unit u's next P
            bool fine = true;
            auto loaded = [&](uint32_t u) {
                fine = fine && barrier_wait(full + 8 * (u % S::kStages), u / S::kStages & 1u, &stalled);
                tmem_fence_after();
            };
            auto written = [&](uint32_t unit) {
                fine = fine && barrier_wait(ready + 8 * unit, given >> unit & 1u, &stalled);
                given ^= 1u << unit;
                tmem_fence_after();
            };
            // S = Q K^T of a unit; frees: whether this was the key tile's last use
            auto score = [&](uint32_t unit, uint32_t queries, uint32_t u, bool frees, bool frees_q, uint32_t buffer) {
                if (fine && elect_one()) {
                    const uint64_t kd = ring_k + (u % S::kStages) * (S::kTileBytes / 16), q = qd + queries * (S::kTileBytes / 16);
#pragma unroll
                    for (int i = 0; i < kDim / 16; ++i) mma_step(tmem + unit * 256, q + row_step(i, kBox), kd + row_step(i, kBox), kScores, i > 0);
                    mma_commit(scored + 8 * unit);
                    if (frees) mma_commit(empty + 8 * (u % S::kStages));
                    if (frees_q) mma_commit(q_empty + 8 * buffer);
                }
                __syncwarp();
            };
            // O += P V of a unit
            auto add = [&](uint32_t unit, uint32_t u, bool first, bool frees, bool last) {
                if (fine && elect_one()) {
                    const uint64_t vd = ring_v + (u % S::kStages) * (S::kTileBytes / 16);
                    const uint32_t at = tmem + unit * 256;
#pragma unroll
                    for (int i = 0; i < kKeys / 16; ++i) mma_step_tmem(at + kKeys, at + i * 8, vd + i * (2048 / 16), kOut, !first || i > 0);
                    if (kTwoTerms)
#pragma unroll
                        for (int i = 0; i < kKeys / 16; ++i) mma_step_tmem(at + kKeys, at + kKeys / 2 + i * 8, vd + i * (2048 / 16), kOut, true);
                    if (frees) mma_commit(empty + 8 * (u % S::kStages));
                    if (last) mma_commit(done + 8 * unit);
                }
                __syncwarp();
            };
            while (fine && cursor.next<kTiles>(p, w)) {
                const uint32_t buffer = piece % S::kQBuffers;
                fine = barrier_wait(q_full + 8 * buffer, piece / S::kQBuffers & 1u, &stalled);
                ++piece;
                tmem_fence_after();
                if (kTiles == 1) {
                    for (int32_t n = 0; n < 2 && n < w.tiles && fine; ++n) {
                        loaded(use);
                        score(n, buffer, use++, true, n == w.tiles - 1, buffer);
                    }
                    for (int32_t n = 0; n < w.tiles && fine; ++n) {
                        loaded(use);
                        written(n & 1);
                        add(n & 1, use++, n < 2, true, n + 2 >= w.tiles);
                        if (n + 2 >= w.tiles) continue;
                        loaded(use);
                        score(n & 1, buffer, use++, true, n + 2 == w.tiles - 1, buffer);
                    }
                } else {
                    const uint32_t last = w.second ? 1 : 0;
                    loaded(use);
                    for (uint32_t u = 0; u <= last; ++u) score(u, u, use, u == last, u == last && w.tiles == 1, buffer);
                    for (int32_t n = 0; n < w.tiles && fine; ++n) {
                        for (uint32_t u = 0; u <= last && fine; ++u) {
                            if (u == 0) loaded(use + 1);
                            written(u);
                            add(u, use + 1, n == 0, u == last, n == w.tiles - 1);
                            if (n + 1 == w.tiles) continue;
                            if (u == 0) loaded(use + 2);
                            score(u, u, use + 2, u == last, u == last && n + 2 == w.tiles, buffer);
                        }
                        use += 2;
                    }
                }
            }
            if (stalled && elect_one()) mma_commit(drained), barrier_drain(drained, 0);
        } else if (warp == kClearWarp) {
            // ---- value rows of the tree: those past it and of absent nodes become zeros, as P's zeros want it;
            // infinities and NaN of the others too, which the rows that see them add at the end
            uint32_t use = 0, piece = 0, turns = 0;  // turns: bit s, the parity of stage s's next tile
            bool fine = true;
            while (fine && cursor.next<kTiles>(p, w)) {
                uint32_t(&odd_nodes)[4] = odd[piece++ % kOddBuffers];
                const int32_t *parents = p.t.parents ? p.t.parents + static_cast<int64_t>(w.b) * a.len_q : nullptr;
                uint32_t there[4];  // (a node below an absent one may count: its values are seen by nobody, and stay finite)
                bool begun = false;
                for (int32_t n = max(0, w.cached / kKeys - w.tile0); n < w.tiles && fine; ++n) {
                    const uint32_t at = use + (kTiles == 2 ? 2 * n + 1 : w.tiles == 1 ? 1 : n < w.tiles - 1 ? 2 * n + 2 : 2 * n + 1);
                    const uint32_t stage = at % S::kStages;
                    if (!begun) {
                        begun = true;
                        if (lane < 4) odd_nodes[lane] = 0;
                        int32_t parent[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int32_t node = 32 * c + static_cast<int32_t>(lane);
                            parent[c] = node >= a.len_q ? -2 : parents ? __ldg(parents + node) : node - 1;
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            there[c] = __ballot_sync(0xFFFFFFFFu, parent[c] >= -1 && parent[c] < 32 * c + static_cast<int32_t>(lane));
                    }
                    fine = barrier_wait(tail + 8 * stage, turns >> stage & 1u, &stalled);
                    turns ^= 1u << stage;
                    if (!fine) break;
                    const int32_t j0 = (w.tile0 + n) * kKeys;
                    uint8_t *rows = smem + S::kRing + stage * S::kTileBytes;
#pragma unroll 2
                    for (int32_t j = max(0, w.cached - j0) + static_cast<int32_t>(lane / 8); j < kKeys; j += 4) {  // a row to 8 lanes
                        const int32_t node = j0 + j - w.cached;
                        const uint32_t word = node < 64 ? node < 32 ? there[0] : there[1] : node < 96 ? there[2] : there[3];
                        const bool gone = node >= kMaxNodes || !(word >> node % 32 & 1u);
                        bool infinite = false;
#pragma unroll
                        for (int c = 0; c < S::kBoxes; ++c) {
                            uint4 *at16 = reinterpret_cast<uint4 *>(rows + c * kBox + j * 128 + lane % 8 * 16);
                            uint4 x = gone ? make_uint4(0, 0, 0, 0) : *at16;
                            constexpr uint32_t kExponent = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
                            uint32_t *half = &x.x;
                            bool change = gone;
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                if ((half[h] & kExponent) == kExponent) half[h] &= 0xFFFF0000u, change = infinite = true;
                                if ((half[h] >> 16 & kExponent) == kExponent) half[h] &= 0xFFFFu, change = infinite = true;
                            }
                            if (change) *at16 = x;
                        }
                        if (infinite) atomicOr(&odd_nodes[node / 32], 1u << node % 32);
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (elect_one()) barrier_arrive(full + 8 * stage);
                }
                use += 2 * w.tiles;
            }
        }
    } else {
        take_registers<kUnitRegisters>();
        // ---- the units' rows
        const int unit = warp / 4;
        const int32_t r = (warp % 4) * 32 + lane, local_node = r / p.pack, head_at = r - local_node * p.pack;
        const uint32_t mine = tmem + unit * 256 + ((warp % 4) * 32u << 16), out = mine + kKeys;
        const float to_base2 = kBias ? kLog2e : a.scale * kLog2e;
        Bits(&seen)[kMaxNodes] = seen_by[unit];
        int16_t(&depth)[kMaxNodes] = depth_by[unit];
        float *values = reinterpret_cast<float *>(smem + S::kTable) + unit * kTableValues;
        const uint8_t *bucket = smem + S::kBuckets;
        const int32_t far = a.table ? a.buckets.max_distance : 0;
        int32_t tree_of = -1, values_of = -1;  // whose `seen` and `values` are there
        uint32_t turn = 0, finished = 0, piece = 0, parts = 0;
        const bool has_bias = kBias && a.table;
        while (cursor.next<kTiles>(p, w)) {
            const int32_t node0 = w.node0 + (kTiles == 2 ? unit * p.nodes_per : 0), i = node0 + local_node, head = w.head0 + head_at;
            const bool valid = local_node < p.nodes_per && i < a.len_q;
            const bool any = __any_sync(0xFFFFFFFFu, valid);
            const bool tree = (w.tile0 + w.tiles) * kKeys > w.cached;  // whether the piece has rows of the tree
            const int64_t index = (static_cast<int64_t>(w.b) * a.heads + head) * a.len_q + i;
            if ((tree || has_bias) && tree_of != w.b) {
                tree_of = w.b;
                sync_threads<128>(2 + unit);
                if (r < a.len_q) {
                    const int32_t *parents = p.t.parents ? p.t.parents + static_cast<int64_t>(w.b) * a.len_q : nullptr;
                    Bits line = 0;
                    int32_t n = -1;
                    if (parents) {
                        for (int32_t at = r; at >= 0; ++n) {
                            line |= Bits(1) << at;
                            const int32_t up = __ldg(parents + at);
                            if (up < -1 || up >= at) {
                                line = 0;
                                break;
                            }
                            at = up;
                        }
                    } else {
                        line = ~Bits(0) >> (kMaxNodes - 1 - r), n = r;
                    }
                    seen[r] = line, depth[r] = static_cast<int16_t>(n);
                }
                sync_threads<128>(2 + unit);
            }
            if (has_bias && values_of != w.pack) {
                values_of = w.pack;
                sync_threads<128>(2 + unit);
                for (int32_t t = r; t < a.buckets.total * p.pack; t += kRows)
                    values[t] = to_f32(static_cast<const T *>(a.table)[t / p.pack * a.heads + w.head0 + t % p.pack]);
                sync_threads<128>(2 + unit);
            }
            const Bits line = (tree || has_bias) && valid ? seen[i] : 0;
            const bool absent = (tree || has_bias) && line == 0;
            const int32_t my_depth = has_bias && valid && !absent ? depth[i] : 0;
            const float far_bias = has_bias && valid ? values[bucket[far] * p.pack + head_at] : 0.0f;
            float top = -INFINITY, sum = 0.0f;
            const int32_t count = kTiles == 1 ? (w.tiles + 1 - unit) / 2 : unit == 0 || w.second ? w.tiles : 0;
#pragma unroll 1
            for (int32_t n = 0; n < count; ++n, ++turn) {
                const int32_t j0 = (w.tile0 + (kTiles == 1 ? 2 * n + unit : n)) * kKeys;
                barrier_wait(scored + 8 * unit, turn & 1u, &stalled);
                tmem_fence_after();
                if (any) {
                    uint32_t s[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_load(s[c], mine + 32 * c);
                    tmem_wait_load(s[0], s[1], s[2], s[3]);
                    if (kBias) {
                        const float2 scale = make_float2(a.scale, a.scale);
                        if (!has_bias || w.cached - (j0 + kKeys - 1) >= far) {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 f = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), scale,
                                                          make_float2(far_bias, far_bias));
                                    s[c][e] = __float_as_uint(f.x), s[c][e + 1] = __float_as_uint(f.y);
                                }
                        } else {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const int32_t node = j0 + 32 * c + e - w.cached;
                                    const int32_t d = my_depth - (node < 0 ? node : static_cast<int32_t>(depth[min(node, a.len_q - 1)]));
                                    s[c][e] = __float_as_uint(fmaf(__uint_as_float(s[c][e]), a.scale,
                                                                   values[bucket[min(max(d, 0), far)] * p.pack + (valid ? head_at : 0)]));
                                }
                        }
                    }
                    if (j0 + kKeys > w.cached) {
                        const int32_t shift = w.cached - j0;  // the tree's first row
                        const Bits visible = absent ? Bits(0) : shift >= 0 ? (Bits(1) << shift) - 1 | line << shift : line >> -shift;
                        const uint32_t word[4] = {static_cast<uint32_t>(visible), static_cast<uint32_t>(visible >> 32),
                                                  static_cast<uint32_t>(visible >> 64), static_cast<uint32_t>(visible >> 96)};
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(word[c] >> e & 1u)) s[c][e] = __float_as_uint(-INFINITY);
                    }
                    float most[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        most[c] = __uint_as_float(s[c][0]);
#pragma unroll
                        for (int e = 1; e < 31; e += 2) most[c] = max3(most[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                        most[c] = fmaxf(most[c], __uint_as_float(s[c][31]));
                    }
                    const float tile_top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
                    // a new maximum, and O and the sum brought to it: at the first finite score, or 2^8 above the old one
                    const bool raise = tile_top > top && (top == -INFINITY || (tile_top - top) * to_base2 > 8.0f);
                    if (__any_sync(0xFFFFFFFFu, raise)) {
                        const float fade = raise ? exp2_approx((top - tile_top) * to_base2) : 1.0f;
                        sum *= fade;
                        if (raise) top = tile_top;
                        if (n > 0) {  // (the products that O is made of were issued before this S)
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
                    // exp2((s - top) to_base2): as one multiply-add, or, where a bias may be the type's
                    // lowest value, with the difference taken first
                    const float from = top == -INFINITY ? 0.0f : -top, shift = kBias ? kLift : fmaf(from, to_base2, kLift);
                    const float2 from2 = make_float2(from, from), shift2 = make_float2(shift, shift);
                    const float2 base2 = make_float2(to_base2, to_base2);
                    float2 total = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t q[16], rest[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 v = make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                            if (kBias) v = add2(v, from2);
                            const float2 f = fma2(v, base2, shift2), x = make_float2(exp2_approx(f.x), exp2_approx(f.y));
                            total = add2(total, x);
                            q[e / 2] = pack2<T>(x.x, x.y);
                            if (kTwoTerms) rest[e / 2] = rest2<T>(x, q[e / 2]);
                        }
                        tmem_store(mine + 16 * c, q);
                        if (kTwoTerms) tmem_store(mine + kKeys / 2 + 16 * c, rest);
                    }
                    sum += total.x + total.y;
                    tmem_wait_store();
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(ready + 8 * unit);
            }

            // ---- the piece's result
            if (count) {
                barrier_wait(done + 8 * unit, finished++ & 1u, &stalled);
                tmem_fence_after();
            }
            const bool whole = w.tiles == w.all, two = kTiles == 1 && w.tiles > 1, writes = kTiles == 2 || unit == 0;
            float weight = 1.0f, other = 0.0f;
            if (two) {
                tops[unit][r] = top, sums[unit][r] = sum;
                sync_threads<256>(1);
                const float top1 = tops[unit ^ 1][r], sum1 = sums[unit ^ 1][r], most = fmaxf(top, top1);
                weight = top == -INFINITY ? 0.0f : exp2_approx((top - most) * to_base2);
                other = top1 == -INFINITY ? 0.0f : exp2_approx((top1 - most) * to_base2);
                // (without a maximum, the sum is 0, or NaN where the scores are)
                sum = (top == -INFINITY ? sum : sum * weight) + (top1 == -INFINITY ? sum1 : sum1 * other);
                top = most;
            }
            // whether it sees values that the products did not
            const uint32_t(&odd_nodes)[4] = odd[piece % kOddBuffers];
            bool some_odd = false;
            if (tree && valid && !absent) {
                const Bits which = Bits(odd_nodes[0]) | Bits(odd_nodes[1]) << 32 | Bits(odd_nodes[2]) << 64 | Bits(odd_nodes[3]) << 96;
                some_odd = (which & line) != 0;
            }
            const float to_natural = kBias ? 1.0f : a.scale;
            const int32_t slot = parts == 0 ? 0 : 1;
            float *part = p.part + ((static_cast<int64_t>(blockIdx.x) * 2 + slot) * p.part_rows + (kTiles == 2 ? unit * p.pack * p.nodes_per : 0) + r) * (kDim + 2);
            const float scale = !whole ? 1.0f : sum == 0.0f || absent ? 0.0f : 1.0f / sum;
            T *o_row = static_cast<T *>(a.out) + w.b * a.os.batch + i * a.os.len + head * a.os.head;
            float *hand = reinterpret_cast<float *>(smem + S::kHand) + r;
#pragma unroll 1
            for (int c = 0; c < kDim / 32; ++c) {
                uint32_t o[32] = {};
                if (count && any) {
                    tmem_load(o, out + 32 * c);
                    tmem_wait_load(o);
                }
                if (two) {  // unit 1 hands its part to unit 0
                    if (c) sync_threads<256>(1);
                    if (unit == 1 && any) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) hand[e * kRows] = __uint_as_float(o[e]);
                    }
                    sync_threads<256>(1);
                }
                if (valid && writes) {
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        v[e] = __uint_as_float(o[e]);
                        if (two) v[e] = v[e] * weight + hand[e * kRows] * other;
                        if (sum == 0.0f || absent) v[e] = 0.0f;  // nothing seen
                        v[e] *= scale;
                    }
                    if (some_odd) {
#pragma unroll 1
                        for (int32_t t = 0; t <= i; ++t) {
                            if (!(odd_nodes[t / 32] >> t % 32 & 1u) || !(line >> t & 1u)) continue;
                            const T *value = static_cast<const T *>(a.v) + w.b * a.vs.batch + (w.cached + t) * a.vs.len + w.head_kv * a.vs.head + 32 * c;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float x = 32 * c + e < a.dim ? to_f32(value[e]) : 0.0f;
                                if (!(fabsf(x) < INFINITY)) v[e] += x;
                            }
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            const float(&eight)[8] = *reinterpret_cast<const float(*)[8]>(&v[e]);
                            if (32 * c + e < a.dim) store<T, 8>(o_row + 32 * c + e, eight);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) *reinterpret_cast<float2 *>(part + 32 * c + e) = make_float2(v[e], v[e + 1]);
                    }
                }
            }
            if (valid && writes) {
                if (!whole)
                    part[kDim] = top * to_natural, part[kDim + 1] = absent ? -1.0f : sum;
                else if (a.lse)
                    a.lse[index] = sum == 0.0f || absent ? -INFINITY : top * to_natural + (logf(sum) - kLift * 0.6931471805599453f);
            }
            if (threadIdx.x == 0 && (parts == 0 || !whole))
                p.meta[blockIdx.x * 2 + slot] = make_int4(w.b, w.unit, w.tile0, kIsThere | (whole ? 0 : kIsPart) | (w.tile0 == 0 ? kStarts : 0) |
                                                                                       (w.tile0 + w.tiles == w.all ? kEnds : 0));
            if (threadIdx.x == 0 && parts == 0) p.meta[blockIdx.x * 2 + 1] = make_int4(0, 0, 0, 0);
            ++parts, ++piece;
            // Both units have read O before the next piece's first P is announced; and they leave together, also when a
            // wait of one of them ran out.
            tmem_fence_before();
            if (!(kTiles == 1 ? all_of<256>(1, !stalled) : all_of<128>(2 + unit, !stalled))) break;
        }
        if (threadIdx.x == 0 && parts == 0) p.meta[blockIdx.x * 2] = p.meta[blockIdx.x * 2 + 1] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) tmem_free<512>(tmem);
}

// Puts the parts of the entries together that blocks have cut: a block to a
// block of the above and some rows, a warp to a row.  An entry's last part is the
// first piece of its block; the others are found going back from there.
template <class T, int kDim, int kTiles>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ TreeParams p)
{
    const Attention &a = p.t.a;
    int32_t block = blockIdx.x, slot = 0;
    const int4 last = p.meta[block * 2];
    if (!(last.w & kIsPart) || (last.w & kStarts) || !(last.w & kEnds)) return;
    const uint32_t lane = threadIdx.x;
    const int32_t row = blockIdx.y * 8 + threadIdx.y, pair = last.y % p.pairs;
    const int32_t i = pair * kTiles * p.nodes_per + row / p.pack, head = last.y / p.pairs * p.pack + row % p.pack, b = last.x;
    if (row >= p.part_rows || i >= a.len_q) return;
    constexpr int kEach = kDim / 32;
    constexpr float kLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;
    float top = -INFINITY, sum = 0.0f, o[kEach] = {};
    bool absent = false;
    for (;;) {
        const float2 *at = reinterpret_cast<const float2 *>(p.part + ((static_cast<int64_t>(block) * 2 + slot) * p.part_rows + row) * (kDim + 2));
        const float2 stats = at[kDim / 2];
        absent = absent || stats.y < 0.0f;
        if (stats.y != 0.0f) {
            const float next = fmaxf(top, stats.x), fade = exp2_approx((top - next) * kLog2e), weight = exp2_approx((stats.x - next) * kLog2e);
            sum = (top == -INFINITY ? 0.0f : sum * fade) + stats.y * weight;
#pragma unroll
            for (int k = 0; k < kEach; k += 2) {
                const float2 v = at[lane * (kEach / 2) + k / 2];
                o[k] = (top == -INFINITY ? 0.0f : o[k] * fade) + v.x * weight, o[k + 1] = (top == -INFINITY ? 0.0f : o[k + 1] * fade) + v.y * weight;
            }
            top = next;
        }
        if (p.meta[block * 2 + slot].w & kStarts) break;
        do --block;
        while (block > 0 && !(p.meta[block * 2].w & kIsThere));
        if (block < 0) break;
        slot = p.meta[block * 2 + 1].w & kIsPart ? 1 : 0;
    }
    if (absent) sum = 0.0f;
    const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
    T *out = static_cast<T *>(a.out) + b * a.os.batch + i * a.os.len + head * a.os.head;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (lane * kEach + k < a.dim) out[lane * kEach + k] = from_f32<T>(sum == 0.0f ? 0.0f : o[k] * scale);
    if (a.lse && lane == 0)
        a.lse[(static_cast<int64_t>(b) * a.heads + head) * a.len_q + i] = sum == 0.0f ? -INFINITY : top + (logf(sum) - kLift * 0.6931471805599453f);
}

// How a call is cut.
struct TreePlan {
    int32_t dim, tiles, pack, nodes_per, packs, pairs, part_rows, blocks;
    bool parts;  // whether an entry's keys may be cut
};

TreePlan tree_plan(const Attention &a)
{
    TreePlan f;
    f.dim = a.dim <= 64 ? 64 : 128;
    // heads side by side: the most of a key head's that divide them evenly, fit a tile, and whose biases fit their place
    f.pack = a.group < kRows ? a.group : kRows;
    while (a.group % f.pack || (a.table && f.pack * a.buckets.total > kTableValues)) --f.pack;
    f.nodes_per = kRows / f.pack;
    if (f.nodes_per > a.len_q) f.nodes_per = a.len_q;
    const int32_t tiles = (a.len_q + f.nodes_per - 1) / f.nodes_per;
    f.tiles = tiles == 1 ? 1 : 2;
    f.packs = a.heads / f.pack, f.pairs = (tiles + f.tiles - 1) / f.tiles;
    f.part_rows = f.tiles * f.pack * f.nodes_per;
    const int32_t key_tiles = (a.len_k + kKeys - 1) / kKeys;
    f.parts = key_tiles >= 2 * kLeastPart;
    const int64_t most = static_cast<int64_t>(a.batch) * f.packs * f.pairs * key_tiles;
    f.blocks = most < sm_count() ? static_cast<int32_t>(most) : static_cast<int32_t>(sm_count());
    return f;
}

size_t meta_bytes(const TreePlan &f) { return sizeof(int4) * 2 * f.blocks; }

template <class T, int kDim, int kTiles, bool kBias>
cudaError_t launch(const TreeParams &p, const TreePlan &f, cudaStream_t s)
{
    using S = Shape<kDim, kTiles>;
    const auto kernel = tree_attention_kernel<T, kDim, kTiles, kBias>;
    static std::atomic<bool> done[16];
    const cudaError_t e = allow_shared(kernel, done);
    if (e != cudaSuccess) return e;
    const size_t bytes = 1024 + S::kTable + (kBias ? S::kBuckets - S::kTable + 1040 : 0);
    static_assert(1024 + S::kBuckets + 1040 <= 222 * 1024, "beside the static arrays");
    kernel<<<f.blocks, kThreads, bytes, s>>>(p);
    note_launch();
    if (f.parts) {
        join_kernel<T, kDim, kTiles><<<dim3(f.blocks, (p.part_rows + 7) / 8), dim3(32, 8), 0, s>>>(p);
        note_launch();
    }
    return cudaGetLastError();
}

template <class T, int kDim>
cudaError_t launch(const TreeParams &p, const TreePlan &f, cudaStream_t s)
{
    const bool bias = has_bias(p.t.a);
    if (f.tiles == 1) return bias ? launch<T, kDim, 1, true>(p, f, s) : launch<T, kDim, 1, false>(p, f, s);
    return bias ? launch<T, kDim, 2, true>(p, f, s) : launch<T, kDim, 2, false>(p, f, s);
}

}  // namespace

cudaError_t stalled_waits_tree(uint64_t *count)
{
    return cudaMemcpyFromSymbol(count, g_stalled_waits, sizeof(uint64_t));
}

size_t tree_attention_workspace(const TreeAttention &t)
{
    const Attention &a = t.a;
    if (a.batch == 0 || a.len_q == 0 || a.heads == 0) return 0;
    const TreePlan f = tree_plan(a);
    return meta_bytes(f) + (f.parts ? sizeof(float) * 2 * f.blocks * f.part_rows * (f.dim + 2) : 0);
}

template <class T>
cudaError_t launch_tree_attention(const TreeAttention &t, cudaStream_t s)
{
    const Attention &a = t.a;
    const TreePlan f = tree_plan(a);
    TreeParams p;
    p.t = t;
    p.pack = f.pack, p.nodes_per = f.nodes_per, p.packs = f.packs, p.pairs = f.pairs, p.part_rows = f.part_rows;
    if (static_cast<int64_t>(f.packs) * f.pairs > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.units = f.packs * f.pairs;
    p.meta = static_cast<int4 *>(a.workspace);
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + meta_bytes(f));
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    cudaError_t e = make_heads_map(&p.q, bf16, a.q, a.qs, a.batch, a.len_q, a.heads, a.dim, f.pack, f.nodes_per * f.pack);
    if (e == cudaSuccess) e = make_heads_map(&p.k, bf16, a.k, a.ks, a.batch, a.len_k, a.heads_kv, a.dim, 1, kKeys);
    if (e == cudaSuccess) e = make_heads_map(&p.v, bf16, a.v, a.vs, a.batch, a.len_k, a.heads_kv, a.dim, 1, kKeys);
    if (e != cudaSuccess) return e;
    return f.dim == 64 ? launch<T, 64>(p, f, s) : launch<T, 128>(p, f, s);
}

template cudaError_t launch_tree_attention<__half>(const TreeAttention &, cudaStream_t);
template cudaError_t launch_tree_attention<__nv_bfloat16>(const TreeAttention &, cudaStream_t);

}  // namespace rngk
