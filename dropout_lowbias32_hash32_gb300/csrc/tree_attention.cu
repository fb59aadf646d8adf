// tree_attention.cu -- attention of a tree of drafted tokens over a cache
// (include/rng.h, rng_tree_attention_fwd) on the tensor cores.
//
// The rows of a key head, its query heads' nodes, are packed into tiles of 128,
// so that its keys are read once.  A unit is such a tile with an O in TMEM and two
// warpgroups: two threads to a row, each with half of a tile's 128 keys; they
// exchange the row's maximum of a tile through shared memory.
//   kTiles = 1 (at most 128 rows of a key head, or less work): one unit with two S,
//     so that a tile's products run under the next one's exponentials;
//   kTiles = 2: two units that share the key tiles, with an S each.
// A unit's step is S = Q K^T, P = exp(S - max) written back over S in 16 bits, O +=
// P V.  One warp issues all products, one the TMA loads, one clears value rows that
// nobody may look at, one has the next pieces of work ready: the nodes' lines, the
// biases.
//
// The work is the list of all (batch entry, key head, rows) and their key tiles,
// cut evenly among the blocks by the lengths found on the device.  A block's first
// and last piece may be a part of one entry's keys; join_kernel puts parts together.
//
// P has two 16-bit terms, its value and what the value's rounding left: one would
// add up to half a step of bf16 to every product, as much as the rounding of o
// itself (8 trees of 64 nodes: 2.3e-3 at most off the formula with one, 1.7e-3 for
// o's rounding alone).  All calls have both, so that a request's rounding does not
// depend on its neighbours or on how its work is cut.
//
// A row's maximum is raised, and O rescaled, only when it has grown by more than
// 2^8: P then stays below 2^8, which 16 bits hold as well as 1.
//
// What bounds it, measured:
//   up to 128 rows of a key head, HBM: 32 trees of 16 nodes, 32 heads over 8 key heads
//     of 128, ragged caches of up to 8192 rows: 547 MB in 93 us (6.0 TB/s read), tensor
//     core 51 %, and 8 us for the parts' join; a chain of 5 over 32768 rows: 134 MB in
//     28 us and 8 us.
//   more rows, the chain of product, exponentials, product in each unit: 8 trees of 64
//     nodes over 4099 rows (256 rows of a key head): 47 us for 14 tiles of keys a block,
//     six products of 512 cycles each; tensor core 52 %.
//   short entries, what a piece costs once: 96 trees of 7 nodes over 115 rows and less, 6
//     heads of 40, a bias: 22 us for four pieces a block; one tree of 8 over 301 rows,
//     10.4 us in a graph; of 19000 cycles, 2400 are set-up and 4300 the first piece's
//     lines and biases.
#include <cmath>

#include "tensor_core.cuh"
#include "tensor_map.h"

namespace rngk {
namespace {

constexpr int kRows = 128, kKeys = 128;  // a unit's tile
constexpr uint32_t kBox = 16384;  // bytes of 128 rows of 64 elements
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxNodes = RNG_MAX_TREE_NODES;
constexpr int kTableValues = 512;   // bias values of a pack of heads by bucket in shared memory
constexpr int kNearValues = 4400;   // and by distance
constexpr int kLeastPart = 2;       // key tiles of a part at least
constexpr int kWhole = 6;           // key tiles that are not cut
constexpr int kOddBuffers = 8;

using Bits = unsigned __int128;
static_assert(kMaxNodes == 128, "a node's line is a 128-bit mask");

struct TreeParams {
    CUtensorMap q, k, v;
    TreeAttention t;
    // heads side by side in a tile, nodes of a tile, packs of heads, pairs (kTiles = 1: single ones) of tiles of a pack,
    // packs x pairs, rows of a part
    int32_t pack, nodes_per, packs, pairs, units, part_rows;
    int32_t least;  // key tiles of a part at least
    Divider by_pack, by_pairs, by_group, by_blocks;
    float *part;  // [blocks][2][dim padded + 2][part_rows]: O, max, sum, rows adjacent
    int4 *meta;   // [blocks][2]: batch entry, unit, first key tile, state; NULL where nothing is cut
};

// A part's state.
constexpr int32_t kIsThere = 1, kIsPart = 2, kStarts = 4, kEnds = 8;

template <int kDim, int kTiles>
struct Shape {
    static constexpr int kBoxes = kDim / 64;
    static constexpr int kQBuffers = 3 - kTiles;
    static constexpr int kThreads = 256 * kTiles + 128;  // two warpgroups a unit, and one of the other roles' warps
    // registers: 384 threads start with 168 each, 2 x 208 + 80 <= 3 x 168; 640 with 96, 4 x 104 + 64 = 5 x 96
    static constexpr int kUnitRegisters = kTiles == 1 ? 208 : 104, kOtherRegisters = kTiles == 1 ? 80 : 64;
    static constexpr uint32_t kTmaWarp = 8 * kTiles, kMmaWarp = kTmaWarp + 1, kClearWarp = kTmaWarp + 2;  // and one for the pieces
    static constexpr int kStages = kDim == 64 ? 8 : 4;
    static constexpr uint32_t kTileBytes = kBoxes * kBox;
    static constexpr uint32_t kRing = 2 * kTileBytes;                    // after two tiles of queries
    static constexpr uint32_t kTable = kRing + kStages * kTileBytes;     // bias values of two pieces
    static constexpr uint32_t kNear = kTable + 2 * kTableValues * 4;     // by distance, of one
    static constexpr uint32_t kBuckets = kNear + kNearValues * 4;        // bucket by distance
};

__device__ __forceinline__ int32_t cached_of(const Attention &a, int32_t b)
{
    const int32_t room = a.len_k - a.len_q;
    return a.key_lengths ? min(max(a.key_lengths[b], 0), room) : room;
}
// Distances that a table by distance has: half a tile that is not all past the last bucket's start has
// 64 keys, and nodes up to 127 deep; odd, so that the heads' values of a distance lie in different banks.
__host__ __device__ __forceinline__ int32_t near_reach(const Buckets &b) { return (b.max_distance + kKeys / 2 + kMaxNodes) | 1; }

__device__ __forceinline__ int32_t tiles_for(const Attention &a, int32_t cached) { return (cached + a.len_q + kKeys - 1) / kKeys; }

// A run of one unit's key tiles.
struct Piece {
    int32_t b, unit, tile0, tiles, all;  // all: of the unit
    int32_t cached, pack, head0, head_kv, node0;
    int32_t second;  // (kTiles = 2) whether the second tile has rows
};

// A block's pieces, one after the other.  In the list that is cut, a unit's key
// tiles come after kTiles entries that stand for what a unit costs beside them (its
// first loads and last sums: about 1.2 tiles' time, 2 where tiles of rows share
// them).
struct Cursor {
    uint32_t at, end, base;  // in the list; base: where the batch entry's units begin
    int32_t b, cached, length;  // its cached rows, and entries of one unit

    template <int kTiles>
    __device__ __forceinline__ bool next(const TreeParams &p, Piece &w)
    {
        if (at >= end) return false;
        const Attention &a = p.t.a;
        while (at >= base + static_cast<uint32_t>(length) * p.units) {
            base += static_cast<uint32_t>(length) * p.units;
            cached = uniform(cached_of(a, ++b));
            length = tiles_for(a, cached) + kTiles;
        }
        const uint32_t local = at - base;
        w.unit = static_cast<int32_t>(local / static_cast<uint32_t>(length));
        const int32_t from = static_cast<int32_t>(local) - w.unit * length, to = min(length, from + static_cast<int32_t>(end - at));
        at += to - from;
        w.b = b, w.cached = cached, w.all = length - kTiles;
        w.tile0 = max(from - kTiles, 0), w.tiles = to - kTiles - w.tile0;
        int32_t pair;
        p.by_pairs.divide(w.unit, w.pack, pair);
        w.head0 = w.pack * p.pack, w.head_kv = p.by_group.quotient(w.head0);
        w.node0 = pair * kTiles * p.nodes_per;
        w.second = kTiles == 2 && w.node0 + p.nodes_per < a.len_q;
        return true;
    }
};

// Where the list is cut at x: at a unit's own beginning or end rather than less than `least` tiles from it.
template <int kTiles>
__device__ __forceinline__ uint32_t snapped(uint32_t x, uint32_t base, uint32_t length, uint32_t least)
{
    const uint32_t o = (x - base) % length;
    return o < kTiles + least ? x - o : length - o < least ? x - o + length : x;
}

// The lines of a tree's nodes (the node and those before it; none for an absent one) and the number of nodes before
// each, by a warp, from the lane's nodes' parents (node lane, lane + 32, ...): each step doubles how far up a line
// reaches.
constexpr int kLaneNodes = kMaxNodes / 32;
__device__ __forceinline__ void find_lines(bool chain, int32_t (&up)[kLaneNodes], Bits (&seen)[kMaxNodes], int16_t (&depth)[kMaxNodes],
                                           int16_t (&jump)[kMaxNodes], uint32_t lane)
{
    constexpr int kEach = kLaneNodes;
    Bits line[kEach];
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
        const int32_t node = 32 * c + static_cast<int32_t>(lane);
        if (up[c] < -1 || up[c] >= node) up[c] = -2;
        line[c] = chain ? ~Bits(0) >> (kMaxNodes - 1 - node) : up[c] == -2 ? Bits(0) : Bits(1) << node;
    }
    bool further = !chain;
#pragma unroll 1
    while (further) {
        further = false;
#pragma unroll
        for (int c = 0; c < kEach; ++c) seen[32 * c + lane] = line[c], jump[32 * c + lane] = static_cast<int16_t>(up[c]);
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kEach; ++c) {
            if (up[c] < 0) continue;
            const Bits more = seen[up[c]];
            line[c] = more ? line[c] | more : Bits(0);
            up[c] = jump[up[c]];
            further = further || up[c] >= 0;
        }
        further = __any_sync(0xFFFFFFFFu, further);
        __syncwarp();  // the next stores come after other lanes' loads (a vote orders no memory)
    }
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
        seen[32 * c + lane] = line[c];
        depth[32 * c + lane] = static_cast<int16_t>(__popcll(static_cast<uint64_t>(line[c])) + __popcll(static_cast<uint64_t>(line[c] >> 64)) - 1);
    }
}

__device__ __forceinline__ void swap_two(int32_t (&v)[2])
{
    const int32_t t = v[0];
    v[0] = v[1], v[1] = t;
}

template <class T, int kDim, int kTiles, bool kBias>
__global__ void __launch_bounds__(Shape<kDim, kTiles>::kThreads, 1) tree_attention_kernel(const __grid_constant__ TreeParams p)
{
    using S = Shape<kDim, kTiles>;
    constexpr int kThreads = S::kThreads;
    constexpr int kLead = kTiles == 1 ? 2 : 1;  // tiles whose S there is room for
    constexpr int kTogether = kBias ? 256 * kTiles : 256;  // threads that begin a piece together
    // f16 holds 2^15: P below 2^8 is lifted, so that long rows' small ones keep their bits
    constexpr float kLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;
    constexpr uint32_t kBars = 3 * S::kStages + 11;  // that one arrival completes
    extern __shared__ uint8_t dynamic[];
    __shared__ alignas(8) uint64_t bars[kBars + 4];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t stalled;
    __shared__ Cursor shared_cursor;
    __shared__ uint32_t scan[kThreads / 32], cut_end;
    __shared__ Piece pieces[2];
    __shared__ Bits seen[2][kMaxNodes];                      // [piece's parity][node]: the nodes of its line
    __shared__ int16_t depth[2][kMaxNodes], jump[kMaxNodes];  // nodes before it
    __shared__ uint32_t odd[kOddBuffers][4];                 // nodes with an infinity or NaN among their values
    __shared__ float tops[2][kTiles][2][kRows], sums[kTiles][2][kRows];  // [tile's parity][unit][half][row]
    const Attention &a = p.t.a;
    const uint32_t warp = uniform(threadIdx.x / 32u), lane = threadIdx.x % 32u;
    uint8_t *smem = dynamic + ((1024u - (smem_address(dynamic) & 1023u)) & 1023u);
    const uint32_t base = smem_address(smem);

    const uint32_t full = smem_address(bars), empty = full + 8 * S::kStages, tail = empty + 8 * S::kStages,
                   scored = tail + 8 * S::kStages, added = scored + 16, q_full = added + 16, q_empty = q_full + 16,
                   drained = q_empty + 16, prepared = drained + 8, ready = prepared + 16, taken = ready + 16;
    if (threadIdx.x < kBars + 4) {
        barrier_init(full + 8 * threadIdx.x, threadIdx.x < kBars ? 1 : 8 * (threadIdx.x < kBars + 2 ? 1 : kTiles));
        fence_barrier_init();
    } else if (threadIdx.x == 64) {
        stalled = 0;
        prefetch_map(&p.q), prefetch_map(&p.k), prefetch_map(&p.v);
    }
    if (warp == S::kMmaWarp) tmem_alloc<512>(smem_address(&tmem_base));
    if (kBias && a.table) {
        uint8_t *bucket = smem + S::kBuckets;
        for (int32_t d = threadIdx.x; d <= a.buckets.max_distance; d += kThreads) bucket[d] = static_cast<uint8_t>(bucket_of(a.buckets, -d));
    }

    // ---- the block's share of the list
    auto block_sum = [&](uint32_t v, uint32_t &before) {  // over the threads; before: over those before this one
        uint32_t up_to = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, up_to, d);
            if (lane >= static_cast<uint32_t>(d)) up_to += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = up_to;
        __syncthreads();
        const uint32_t w = lane < kThreads / 32 ? scan[lane] : 0;
        before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0) + up_to - v;
        return __reduce_add_sync(0xFFFFFFFFu, w);
    };
    {
        const int32_t mine = threadIdx.x;
        uint32_t sum = 0, before, so_far = 0;
        int32_t cached = 0;
        for (int32_t b = mine; b < a.batch; b += kThreads) cached = cached_of(a, b), sum += tiles_for(a, cached) + kTiles;
        const uint32_t all = block_sum(sum, before) * p.units;
        const uint32_t share = p.by_blocks.quotient(all), left = all - share * p.by_blocks.by;
        // at every all / blocks, rounded down
        auto cut = [&](uint32_t block) { return block * share + p.by_blocks.quotient(block * left); };
        const uint32_t from = cut(blockIdx.x), to = cut(blockIdx.x + 1);
        if (threadIdx.x == 0) shared_cursor = Cursor{all, all, all, a.batch - 1, 0, 1}, cut_end = all;
        for (int32_t b0 = 0; b0 < a.batch; b0 += kThreads) {
            const int32_t b = b0 + mine;
            if (a.batch > kThreads) {  // (else the first sum had one entry to a thread)
                sum = b < a.batch ? cached = cached_of(a, b), tiles_for(a, cached) + kTiles : 0;
                const uint32_t part = block_sum(sum, before);
                before += so_far, so_far += part;
            } else {
                __syncthreads();
            }
            const uint32_t begin = before * p.units, past = begin + sum * p.units;
            if (from >= begin && from < past) shared_cursor = Cursor{snapped<kTiles>(from, begin, sum, p.least), 0, begin, b, cached, static_cast<int32_t>(sum)};
            if (to >= begin && to < past) cut_end = snapped<kTiles>(to, begin, sum, p.least);
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = uniform(tmem_base);
    Cursor cursor{uniform(shared_cursor.at), uniform(cut_end), uniform(shared_cursor.base), uniform(shared_cursor.b),
                  uniform(shared_cursor.cached), uniform(shared_cursor.length)};
    Piece w;
    grid_let_next();

    if (warp >= S::kTmaWarp) {
        give_registers<S::kOtherRegisters>();
        if (warp == S::kTmaWarp) {
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
#pragma unroll 1  // K_0 .. K_{lead-1}, then V_n and K_{n+lead}
                for (int32_t n = -2 * kLead; n < 2 * w.tiles; ++n) {
                    const bool value = n >= 0 && n % 2 == 0;
                    const int32_t tile = n / 2 + (value ? 0 : kLead);
                    if ((n < 0 && n % 2 != 0) || tile >= w.tiles) continue;
                    const uint32_t stage = use % S::kStages, dst = base + S::kRing + stage * S::kTileBytes;
                    fine = barrier_wait(empty + 8 * stage, (use / S::kStages & 1u) ^ 1u, &stalled);
                    if (!fine) break;
                    ++use;
                    // value rows from the tree on are looked through before the products see them
                    const bool looked_through = value && (w.tile0 + tile + 1) * kKeys > w.cached;
                    const uint32_t bar = (looked_through ? tail : full) + 8 * stage;
                    on_tail = looked_through ? on_tail | 1u << stage : on_tail & ~(1u << stage);
                    tail_turns ^= looked_through ? 1u << stage : 0u;
                    if (elect_one()) {
                        barrier_expect(bar, S::kTileBytes);
#pragma unroll
                        for (int c = 0; c < S::kBoxes; ++c)
                            tma_load_5d(dst + c * kBox, value ? &p.v : &p.k, bar, c * 64, 0, (w.tile0 + tile) * kKeys, w.head_kv, w.b);
                    }
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
        } else if (warp == S::kMmaWarp) {
            // ---- MMA
            constexpr int kUnrolled = kTiles == 1 ? 1 : 8;
            constexpr uint32_t kScores = mma_shape<T>(kKeys, false), kOut = mma_shape<T>(kDim, true);
            const uint64_t ring_v = column_major_tile(base + S::kRing, S::kBoxes > 1 ? kBox : 1024);
            const uint64_t ring_k = row_major_tile(base + S::kRing), qd = row_major_tile(base);
            uint32_t use = 0, piece = 0, given = 0;  // given: bit s, the parity of S s's next P
            bool fine = true;
            auto loaded = [&](uint32_t u) {
                fine = fine && barrier_wait(full + 8 * (u % S::kStages), u / S::kStages & 1u, &stalled);
                tmem_fence_after();
            };
            // S = Q K^T
            auto score = [&](uint32_t which, uint32_t queries, uint32_t u, bool frees, bool frees_q, uint32_t buffer) {
                if (fine && elect_one()) {
                    const uint64_t kd = ring_k + (u % S::kStages) * (S::kTileBytes / 16), q = qd + queries * (S::kTileBytes / 16);
#pragma unroll(kUnrolled)
                    for (int i = 0; i < kDim / 16; ++i) mma_step(tmem + which * kKeys, q + row_step(i, kBox), kd + row_step(i, kBox), kScores, i > 0);
                    mma_commit(scored + 8 * which);
                    if (frees) mma_commit(empty + 8 * (u % S::kStages));
                    if (frees_q) mma_commit(q_empty + 8 * buffer);
                }
                __syncwarp();
            };
            // O += P V over `steps` of 16 keys; P lies where the scores were, 16 columns for 32 keys, and beside them its
            // second term
            auto add = [&](uint32_t which, uint32_t unit, uint32_t u, int32_t steps, bool first, bool frees) {
                if (fine && elect_one()) {
                    const uint64_t vd = ring_v + (u % S::kStages) * (S::kTileBytes / 16);
                    const uint32_t at = tmem + which * kKeys, o = tmem + (2 + unit) * kKeys;
#pragma unroll(kUnrolled)
                    for (int i = 0; i < kKeys / 16; ++i) {
                        if (i >= steps) break;
                        const uint32_t from = at + (i / 2) * 32 + i % 2 * 8;
                        mma_step_tmem(o, from, vd + i * (2048 / 16), kOut, !first || i > 0);
                        mma_step_tmem(o, from + 16, vd + i * (2048 / 16), kOut, true);
                    }
                    if (frees) mma_commit(empty + 8 * (u % S::kStages));
                    mma_commit(added + 8 * unit);
                }
                __syncwarp();
            };
            while (fine && cursor.next<kTiles>(p, w)) {
                const uint32_t buffer = piece % S::kQBuffers;
                fine = barrier_wait(q_full + 8 * buffer, piece / S::kQBuffers & 1u, &stalled);
                ++piece;
                tmem_fence_after();
                // a step: the sums of tile n (from 0 on), then the scores of the one that takes its place
                const uint32_t last = w.second ? 1 : 0;
                const int32_t keys = w.cached + a.len_q - w.tile0 * kKeys;
#pragma unroll 1
                for (int32_t n = -kLead; n < w.tiles && fine; ++n) {
                    const int32_t next = n + kLead;
                    const uint32_t value = use, key = use + (n >= 0 ? 1 : 0);
                    if (n < 0 && next >= w.tiles) continue;
#pragma unroll 1
                    for (uint32_t u = 0; u <= last && fine; ++u) {
                        const uint32_t which = kTiles == 1 ? n & 1 : u;
                        if (n >= 0) {
                            if (u == 0) loaded(value);
                            fine = fine && barrier_wait(ready + 8 * which, given >> which & 1u, &stalled);
                            given ^= 1u << which;
                            tmem_fence_after();
                            add(which, u, value, (keys - n * kKeys + 15) / 16, n == 0, u == last);
                        }
                        if (next >= w.tiles) continue;
                        if (u == 0) loaded(key);
                        score(which, kTiles == 1 ? buffer : u, key, u == last, u == last && next == w.tiles - 1, buffer);
                    }
                    use += (n >= 0 ? 1 : 0) + (next < w.tiles ? 1 : 0);
                }
            }
            if (stalled && elect_one()) mma_commit(drained), barrier_drain(drained, 0);
        } else if (warp == S::kClearWarp) {
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
                        __syncwarp();
                    }
                    fine = barrier_wait(tail + 8 * stage, turns >> stage & 1u, &stalled);
                    turns ^= 1u << stage;
                    if (!fine) break;
                    const int32_t j0 = (w.tile0 + n) * kKeys, end = min(kKeys, (w.cached + a.len_q - j0 + 15) / 16 * 16);  // what the products take
                    uint8_t *rows = smem + S::kRing + stage * S::kTileBytes;
                    // a finite number's bits without its sign, plus this, stay below 2^15
                    constexpr uint32_t kToSign = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
                    constexpr int kAtOnce = 4;
                    auto over = [&](uint32_t y) { return (y & 0x7FFF7FFFu) + kToSign; };
                    auto finite = [&](uint32_t y) {
                        const uint32_t o = over(y);
                        return y & ~((o & 0x8000u ? 0xFFFFu : 0u) | (o & 0x80000000u ? 0xFFFF0000u : 0u));
                    };
                    uint8_t *at16 = rows + lane % 8 * 16;  // a row to 8 lanes
#pragma unroll 1
                    for (int32_t j4 = max(0, w.cached - j0) + static_cast<int32_t>(lane / 8); j4 < end; j4 += 4 * kAtOnce) {
                        uint4 x[kAtOnce][S::kBoxes];
#pragma unroll
                        for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
                            for (int c = 0; c < S::kBoxes; ++c)
                                x[u][c] = *reinterpret_cast<const uint4 *>(at16 + c * kBox + min(j4 + 4 * u, kKeys - 1) * 128);
#pragma unroll
                        for (int u = 0; u < kAtOnce; ++u) {
                            const int32_t j = j4 + 4 * u, node = j0 + j - w.cached;
                            const uint32_t word = node < 64 ? node < 32 ? there[0] : there[1] : node < 96 ? there[2] : there[3];
                            const bool gone = node >= kMaxNodes || !(word >> node % 32 & 1u);
                            bool infinite = false;
#pragma unroll
                            for (int c = 0; c < S::kBoxes; ++c) {
                                const uint4 y = x[u][c];
                                infinite = infinite || ((over(y.x) | over(y.y) | over(y.z) | over(y.w)) & 0x80008000u);
                            }
                            if (j >= end || !(gone || infinite)) continue;
#pragma unroll
                            for (int c = 0; c < S::kBoxes; ++c) {
                                const uint4 y = x[u][c];
                                *reinterpret_cast<uint4 *>(at16 + c * kBox + j * 128) =
                                    gone ? make_uint4(0, 0, 0, 0) : make_uint4(finite(y.x), finite(y.y), finite(y.z), finite(y.w));
                            }
                            if (!gone) atomicOr(&odd_nodes[node / 32], 1u << node % 32);
                        }
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (elect_one()) barrier_arrive(full + 8 * stage);
                }
                use += 2 * w.tiles;
            }
        } else {
            // ---- the next pieces: two are ready
            const bool has_bias = kBias && a.table;
            int32_t lines_of[2] = {-1, -1}, values_of[2] = {-1, -1};
            for (uint32_t piece = 0;; ++piece) {
                const uint32_t buffer = piece & 1u;
                const bool more = cursor.next<kTiles>(p, w);
                if (piece >= 2 && !barrier_wait(taken + 8 * buffer, (piece / 2 - 1) & 1u, &stalled)) break;
                if (!more) w.tiles = 0;
                if (lane == 0) pieces[buffer] = w;
                const bool tree = (w.tile0 + w.tiles) * kKeys > w.cached;  // whether the piece has rows of the tree
                const bool lines = more && (tree || has_bias) && lines_of[0] != w.b, biases = more && has_bias && values_of[0] != w.pack;
                // all loads first
                int32_t up[kLaneNodes];
                if (lines) {
                    const int32_t *parents = p.t.parents ? p.t.parents + static_cast<int64_t>(w.b) * a.len_q : nullptr;
#pragma unroll
                    for (int k = 0; k < kLaneNodes; ++k) {
                        const int32_t node = 32 * k + static_cast<int32_t>(lane);
                        up[k] = parents && node < a.len_q ? __ldg(parents + node) : -2;
                    }
                }
                constexpr int kAtOnce = 4;
                float *values = reinterpret_cast<float *>(smem + S::kTable) + buffer * kTableValues;
                auto value_at = [&](int32_t t) {
                    int32_t n, head;
                    p.by_pack.divide(t, n, head);
                    return static_cast<const T *>(a.table)[n * a.heads + w.head0 + head];
                };
                const int32_t count = biases ? a.buckets.total * p.pack : 0;
                T first[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (static_cast<int32_t>(lane) + 32 * k < count) first[k] = value_at(lane + 32 * k);
                if (lines) {
                    lines_of[0] = w.b;
                    find_lines(!p.t.parents, up, seen[buffer], depth[buffer], jump, lane);
                }
                if (biases) {
                    values_of[0] = w.pack;
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k)
                        if (static_cast<int32_t>(lane) + 32 * k < count) values[lane + 32 * k] = to_f32(first[k]);
                    for (int32_t t = lane + 32 * kAtOnce; t < count; t += 32) values[t] = to_f32(value_at(t));
                }
                swap_two(lines_of), swap_two(values_of);  // [0]: of the buffer that comes next
                __syncwarp();
                if (lane == 0) barrier_arrive(prepared + 8 * buffer);
                if (!more) break;
            }
        }
    } else {
        take_registers<S::kUnitRegisters>();
        // ---- the units' rows
        const int unit = warp / 8, half = warp / 4 % 2;
        const int32_t r = (warp % 4) * 32 + lane;
        int32_t local_node, head_at;
        p.by_pack.divide(r, local_node, head_at);
        const uint32_t lanes = tmem + ((warp % 4) * 32u << 16), out = lanes + (2 + unit) * kKeys + half * (kDim / 2);
        const int pair = 1 + kTiles + unit * 4 + warp % 4;  // the barrier of the two warps that share rows
        const float to_base2 = kBias ? kLog2e : a.scale * kLog2e;
        const uint8_t *bucket = smem + S::kBuckets;
        const bool has_bias = kBias && a.table;
        const int32_t far = has_bias ? a.buckets.max_distance : 0, reach = has_bias ? near_reach(a.buckets) : 0;
        float *near_table = reinterpret_cast<float *>(smem + S::kNear);
        int32_t near_of = -1;  // whose biases it holds
        uint32_t turns = 0, additions = 0, parts = 0;  // turns: bit s, the parity of S s's next tile
#pragma unroll 1
        for (uint32_t piece = 0;; ++piece) {
            // They leave together, also when a wait of one of them ran out.
            tmem_fence_before();
            const uint32_t buffer = piece & 1u;
            const bool fine = barrier_wait(prepared + 8 * buffer, piece / 2 & 1u, &stalled);
            if (!all_of<kTogether>(kBias ? 1 : 1 + unit, fine && !stalled)) break;
            w = pieces[buffer];
            if (w.tiles == 0) break;
            const float *values = reinterpret_cast<const float *>(smem + S::kTable) + buffer * kTableValues;
            if (has_bias && near_of != w.pack && w.cached - ((w.tile0 + w.tiles) * kKeys - 1) < far) {
                near_of = w.pack;
                for (int32_t d = threadIdx.x; d < reach; d += kTogether) {
                    const float *by_head = values + bucket[min(d, far)] * p.pack;
                    for (int32_t h = 0; h < p.pack; ++h) near_table[h * reach + d] = by_head[h];
                }
                sync_threads<kTogether>(1);
            }
            const int32_t i = w.node0 + (kTiles == 2 ? unit * p.nodes_per : 0) + local_node, head = w.head0 + head_at;
            const bool valid = local_node < p.nodes_per && i < a.len_q;
            const bool any = __any_sync(0xFFFFFFFFu, valid);
            const bool tree = (w.tile0 + w.tiles) * kKeys > w.cached;  // whether the piece has rows of the tree
            const int64_t index = (static_cast<int64_t>(w.b) * a.heads + head) * a.len_q + i;
            const Bits line = (tree || has_bias) && valid ? seen[buffer][i] : 0;
            const bool absent = (tree || has_bias) && line == 0;
            const int32_t my_depth = has_bias && valid ? depth[buffer][i] : 0;
            const float far_bias = has_bias ? values[bucket[far] * p.pack + (valid ? head_at : 0)] : 0.0f;
            const float *near_bias = near_table + (valid ? head_at : 0) * reach;
            float top = -INFINITY, sum = 0.0f;
            const int32_t count = unit == 0 || w.second ? w.tiles : 0;
#pragma unroll 1
            for (int32_t n = 0; n < count; ++n) {
                const uint32_t which = kTiles == 1 ? n & 1 : unit;
                const uint32_t mine = lanes + which * kKeys + half * (kKeys / 2);
                const int32_t j0 = (w.tile0 + n) * kKeys + half * (kKeys / 2);  // this half's
                barrier_wait(scored + 8 * which, turns >> which & 1u, &stalled);
                turns ^= 1u << which;
                tmem_fence_after();
                if (any) {
                    const bool near = has_bias && w.cached - (j0 + kKeys / 2 - 1) < far, masked = j0 + kKeys / 2 > w.cached;
                    const int32_t shift = w.cached - j0;  // the tree's first row
                    uint64_t visible = ~uint64_t(0);
                    if (masked)
                        visible = static_cast<uint64_t>(absent ? Bits(0) : shift >= 0 ? ((Bits(1) << shift) - 1) | line << shift : shift > -kMaxNodes ? line >> -shift : Bits(0));
                    uint32_t s[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_load(s[c], mine + 32 * c);
                    tmem_wait_load(s[0], s[1]);
                    if (kBias) {
                        const float2 scale = make_float2(a.scale, a.scale);
                        if (!near) {
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 f = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), scale,
                                                          make_float2(far_bias, far_bias));
                                    s[c][e] = __float_as_uint(f.x), s[c][e + 1] = __float_as_uint(f.y);
                                }
                        } else {
                            const float *back = near_bias + my_depth + shift;  // of the first key; the next ones are nearer
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                if (32 * c + 32 <= shift) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        s[c][e] = __float_as_uint(fmaf(__uint_as_float(s[c][e]), a.scale, back[-(32 * c + e)]));
                                } else {  // some of the tree: a key's place among them from the lane that has looked it up
                                    const int32_t key = 32 * c + static_cast<int32_t>(lane) - shift;
                                    int32_t place = depth[buffer][min(max(key, 0), a.len_q - 1)];
                                    place = key < 0 ? key : place;
#pragma unroll
                                    for (int e = 0; e < 32; ++e) {
                                        const int32_t d = max(my_depth - __shfl_sync(0xFFFFFFFFu, place, e), 0);
                                        s[c][e] = __float_as_uint(fmaf(__uint_as_float(s[c][e]), a.scale, near_bias[d]));
                                    }
                                }
                            }
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t word = static_cast<uint32_t>(visible >> 32 * c);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(word >> e & 1u)) s[c][e] = __float_as_uint(-INFINITY);
                        }
                    }
                    float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            most[0] = max3(most[0], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                            most[1] = max3(most[1], __uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3]));
                        }
                    // the row's maximum, of both halves
                    float(&shared_tops)[2][kRows] = tops[n & 1][unit];
                    float tile_top = fmaxf(most[0], most[1]);
                    shared_tops[half][r] = tile_top;
                    sync_threads<64>(pair);
                    tile_top = fmaxf(tile_top, shared_tops[half ^ 1][r]);
                    // a new maximum, and O and the sum brought to it: at the first finite score, or 2^8 above the old one
                    const bool raise = tile_top > top && (top == -INFINITY || (tile_top - top) * to_base2 > 8.0f);
                    if (__any_sync(0xFFFFFFFFu, raise)) {
                        const float fade = raise ? exp2_approx((top - tile_top) * to_base2) : 1.0f;
                        sum *= fade;
                        if (raise) top = tile_top;
                        if (n > 0) {
                            // O up to the previous tile (kTiles = 2: its products were issued before this S)
                            if (kTiles == 1) barrier_wait(added, (additions + n - 1) & 1u, &stalled);
                            tmem_fence_after();
#pragma unroll 1
                            for (int c = 0; c < kDim / 32; ++c) {
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
                    const float from = top == -INFINITY ? 0.0f : -top, shift_2 = kBias ? kLift : fmaf(from, to_base2, kLift);
                    const float2 from2 = make_float2(from, from), shift2 = make_float2(shift_2, shift_2);
                    const float2 base2 = make_float2(to_base2, to_base2);
                    float2 total = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {  // 16 columns at a time
                        uint32_t q[8], rest[8];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const uint32_t(&two)[2] = *reinterpret_cast<const uint32_t(*)[2]>(&s[c / 2][c % 2 * 16 + e]);
                            float2 v = make_float2(__uint_as_float(two[0]), __uint_as_float(two[1]));
                            if (kBias) v = add2(v, from2);
                            const float2 f = fma2(v, base2, shift2), x = make_float2(exp2_approx(f.x), exp2_approx(f.y));
                            total = add2(total, x);
                            q[e / 2] = pack2<T>(x.x, x.y);
                            rest[e / 2] = rest2<T>(x, q[e / 2]);
                        }
                        const uint32_t to = mine + 32 * (c / 2) + 8 * (c % 2);
                        tmem_store(to, q);
                        tmem_store(to + 16, rest);
                    }
                    sum += total.x + total.y;
                    tmem_wait_store();
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(ready + 8 * which);
            }
            if (lane == 0) barrier_arrive(taken + 8 * buffer);

            // ---- the piece's result
            sums[unit][half][r] = sum;
            sync_threads<64>(pair);
            sum += sums[unit][half ^ 1][r];
            if (count) {
                additions += count;
                // (one after the other: a wait tells a phase from the next one only)
                if (kTiles == 1 && count > 1) barrier_wait(added, (additions - 2) & 1u, &stalled);
                barrier_wait(added + 8 * unit, (additions - 1) & 1u, &stalled);
                tmem_fence_after();
            }
            const bool whole = w.tiles == w.all;
            // whether it sees values that the products did not
            const uint32_t(&odd_nodes)[4] = odd[piece % kOddBuffers];
            bool some_odd = false;
            if (tree && valid && !absent) {
                const Bits which = Bits(odd_nodes[0]) | Bits(odd_nodes[1]) << 32 | Bits(odd_nodes[2]) << 64 | Bits(odd_nodes[3]) << 96;
                some_odd = (which & line) != 0;
            }
            const float to_natural = kBias ? 1.0f : a.scale;
            const int32_t slot = parts == 0 ? 0 : 1;
            float *part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * p.part_rows * (kDim + 2) + unit * kRows + r;
            const float scale = !whole ? 1.0f : sum == 0.0f || absent ? 0.0f : 1.0f / sum;
            T *o_row = static_cast<T *>(a.out) + w.b * a.os.batch + i * a.os.len + head * a.os.head;
#pragma unroll 1
            for (int c = 0; c < kDim / 64; ++c) {
                const int col = half * (kDim / 2) + 32 * c;
                uint32_t o[32] = {};
                if (count && any) {
                    tmem_load(o, out + 32 * c);
                    tmem_wait_load(o);
                }
                if (!valid) continue;
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    v[e] = __uint_as_float(o[e]);
                    if (sum == 0.0f || absent) v[e] = 0.0f;  // nothing seen
                    v[e] *= scale;
                }
                if (some_odd) {
#pragma unroll 1
                    for (int32_t t = 0; t <= i; ++t) {
                        if (!(odd_nodes[t / 32] >> t % 32 & 1u) || !(line >> t & 1u)) continue;
                        const T *value = static_cast<const T *>(a.v) + w.b * a.vs.batch + (w.cached + t) * a.vs.len + w.head_kv * a.vs.head + col;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = col + e < a.dim ? to_f32(value[e]) : 0.0f;
                            if (!(fabsf(x) < INFINITY)) v[e] += x;
                        }
                    }
                }
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        const float(&eight)[8] = *reinterpret_cast<const float(*)[8]>(&v[e]);
                        if (col + e < a.dim) store<T, 8>(o_row + col + e, eight);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) part[(col + e) * p.part_rows] = v[e];
                }
            }
            if (valid && half == 0) {
                if (!whole)
                    part[kDim * p.part_rows] = top * to_natural, part[(kDim + 1) * p.part_rows] = absent ? -1.0f : sum;
                else if (a.lse)
                    a.lse[index] = sum == 0.0f || absent ? -INFINITY : top * to_natural + (logf(sum) - kLift * 0.6931471805599453f);
            }
            if (p.meta && threadIdx.x == 0 && (parts == 0 || !whole))
                p.meta[blockIdx.x * 2 + slot] = make_int4(w.b, w.unit, w.tile0, kIsThere | (whole ? 0 : kIsPart) | (w.tile0 == 0 ? kStarts : 0) |
                                                                                       (w.tile0 + w.tiles == w.all ? kEnds : 0));
            if (p.meta && threadIdx.x == 0 && parts == 0) p.meta[blockIdx.x * 2 + 1] = make_int4(0, 0, 0, 0);
            ++parts;
        }
        if (p.meta && threadIdx.x == 0 && parts == 0) p.meta[blockIdx.x * 2] = p.meta[blockIdx.x * 2 + 1] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == S::kMmaWarp) tmem_free<512>(tmem);
}

__device__ __forceinline__ float scaled(float x, float by) { return by == 0.0f ? (fabsf(x) < INFINITY ? 0.0f : x) : x * by; }

// Puts the parts of the entries together that blocks have cut: blocks to a block
// of the above and 32 rows, a thread to a row and 8 columns.  An entry's last part
// is the first piece of its block; the others lie in the blocks before it, which a
// warp looks up 32 at a time.  Few rows have many parts, which are read by many
// small blocks, eight parts at once; many rows have few (8 x 64 nodes, 32 over 8
// heads of 128: 28 MB of them).
template <class T, int kDim, int kTiles>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ TreeParams p)
{
    const Attention &a = p.t.a;
    grid_wait();
    const int4 last = p.meta[blockIdx.x * 2];
    if (!(last.w & kIsPart) || (last.w & kStarts) || !(last.w & kEnds)) return;
    constexpr float kLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;
    constexpr int kAtOnce = kTiles == 1 ? 8 : 4, kEach = 8;
    const int32_t lane = threadIdx.x, row = blockIdx.y * 32 + lane, col = (blockIdx.z * blockDim.y + threadIdx.y) * kEach;
    int32_t pack, pair, local_node, head_at;
    p.by_pairs.divide(last.y, pack, pair);
    p.by_pack.divide(row % kRows, local_node, head_at);
    const int32_t i = (pair * kTiles + row / kRows) * p.nodes_per + local_node, head = pack * p.pack + head_at, b = last.x;
    const bool valid = local_node < p.nodes_per && i < a.len_q;
    float top = -INFINITY, sum = 0.0f, o[kEach] = {};
    bool absent = false, started = false;
    for (int32_t block0 = blockIdx.x; !started && block0 >= 0; block0 -= 32) {
        // a lane to a block: the slot of its part of this entry, -1 for none
        const int32_t block = block0 - lane;
        int32_t slot = -1;
        bool starts = false;
        if (block >= 0) {
            const int4 first = p.meta[block * 2], second = p.meta[block * 2 + 1];
            if (block == static_cast<int32_t>(blockIdx.x)) slot = 0;
            else if (second.w & kIsPart) slot = 1, starts = true;
            else if (first.w & kIsThere) slot = 0, starts = first.w & kStarts;
        }
        const uint32_t stops = __ballot_sync(0xFFFFFFFFu, starts);
        started = stops != 0;
        uint32_t there = __ballot_sync(0xFFFFFFFFu, slot >= 0) & (stops ? (2u << (__ffs(stops) - 1)) - 1u : 0xFFFFFFFFu);
        while (there) {
            float stats[kAtOnce][2], v[kAtOnce][kEach];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int32_t which = there ? __ffs(there) - 1 : -1;
                there &= there - 1u;
                const int32_t at_slot = __shfl_sync(0xFFFFFFFFu, slot, which < 0 ? 0 : which);
                const float *at = p.part + (static_cast<int64_t>(block0 - which) * 2 + at_slot) * p.part_rows * (kDim + 2) + row;
                const bool reads = which >= 0 && valid;
                stats[u][0] = reads ? at[kDim * p.part_rows] : -INFINITY, stats[u][1] = reads ? at[(kDim + 1) * p.part_rows] : 0.0f;
#pragma unroll
                for (int k = 0; k < kEach; ++k) v[u][k] = reads ? at[(col + k) * p.part_rows] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                absent = absent || stats[u][1] < 0.0f;
                if (stats[u][1] == 0.0f) continue;
                const float next = fmaxf(top, stats[u][0]), fade = top == -INFINITY ? 1.0f : exp2_approx((top - next) * kLog2e);
                const float weight = exp2_approx((stats[u][0] - next) * kLog2e);
                sum = sum * fade + stats[u][1] * weight;
                top = next;
                // a factor that f32 no longer holds is more than 0 all the same: what is not finite stays
                if (fade == 0.0f || weight == 0.0f) {
#pragma unroll
                    for (int k = 0; k < kEach; ++k) o[k] = scaled(o[k], fade) + scaled(v[u][k], weight);
                    continue;
                }
#pragma unroll
                for (int k = 0; k < kEach; ++k) o[k] = o[k] * fade + v[u][k] * weight;
            }
        }
    }
    if (!valid) return;
    if (absent) sum = 0.0f;
    if (col < a.dim) {
        const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int k = 0; k < kEach; ++k) o[k] = sum == 0.0f ? 0.0f : o[k] * scale;
        store<T, 8>(static_cast<T *>(a.out) + b * a.os.batch + i * a.os.len + head * a.os.head + col, o);
    }
    if (a.lse && col == 0)
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
    while (a.group % f.pack || (a.table && f.pack > 1 && (f.pack * a.buckets.total > kTableValues || f.pack * near_reach(a.buckets) > kNearValues)))
        --f.pack;
    f.nodes_per = kRows / f.pack;
    if (f.nodes_per > a.len_q) f.nodes_per = a.len_q;
    const int32_t tiles = (a.len_q + f.nodes_per - 1) / f.nodes_per;
    const int32_t key_tiles = (a.len_k + kKeys - 1) / kKeys, sms = static_cast<int32_t>(sm_count());
    // The parts' join, a second launch, costs the host as much as the first (call 11.5 us, 22 with it); on the device 6
    // key tiles of 8 heads take 17.5 us uncut, 15.5 cut, with 8 entries 19.6 and 21.6; 12 tiles 23.7 and 19.6, 25.7 and
    // 27.8.
    f.parts = key_tiles > kWhole;
    // Two tiles of rows to a block share what is loaded, and one's products run beside the other's exponentials, but the
    // block's first and last steps take longer.  Uncut, a block with two takes 1.83 times one's time, and whole rounds of
    // the SMs count: 32 heads over 8 of 128, 128 nodes, 700 rows, 16 entries 43.4 us with two and 52.9 with one (2 rounds
    // and 4), 4 entries 24.0 and 16.6 (1 and 1); 64 nodes, 300 rows, 64 entries 56.8 and 50.8 (4 and 7).  Cut, two from
    // ten key tiles a block on, where no half of a pair is idle: 64 nodes, 4 x 4099 rows (6.9) 38.0 and 33.6, 8 x 4099
    // (13.9) 56.2 and 56.5, 32 x 2000 (26.9) 98.5 and 106; 16 heads over one, 40 nodes (five tiles of rows), 32 x 2000 48.4
    // and 41.1.
    f.packs = a.heads / f.pack;
    const double rows = static_cast<double>(a.batch) * f.packs, pairs = (tiles + 1) / 2;
    const bool two = f.parts ? tiles % 2 == 0 && rows * pairs * key_tiles > 10.0 * sms
                             : 1.83 * std::ceil(rows * pairs / sms) < std::ceil(rows * tiles / sms);
    f.tiles = two ? 2 : 1;
    f.pairs = (tiles + f.tiles - 1) / f.tiles;
    f.part_rows = f.tiles == 2 ? 2 * kRows : (f.pack * f.nodes_per + 31) / 32 * 32;
    // the list of key tiles has less than 2^31 entries: more would be 2^38 rows of keys
    const double units = static_cast<double>(a.batch) * f.packs * f.pairs;
    f.blocks = units * (key_tiles + f.tiles) > 0x7FFFFFFF ? 0 : units * key_tiles < sms ? static_cast<int32_t>(units * key_tiles) : sms;
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
    static_assert(1024 + S::kBuckets + 1040 + 11 * 1024 + 512 <= 227 * 1024 || kTiles == 1, "beside the static arrays");
    static_assert(1024 + S::kBuckets + 1040 + 8 * 1024 + 512 <= 227 * 1024, "beside the static arrays");
    kernel<<<f.blocks, S::kThreads, bytes, s>>>(p);
    note_launch();
    if (f.parts) {
        cudaLaunchConfig_t config = {};
        const int warps = p.part_rows <= 32 ? 2 : 8;
        config.gridDim = dim3(f.blocks, p.part_rows / 32, kDim / 8 / warps), config.blockDim = dim3(32, warps), config.stream = s;
        cudaLaunchAttribute early;
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization, early.val.programmaticStreamSerializationAllowed = 1;
        config.attrs = &early, config.numAttrs = 1;
        const cudaError_t joined = cudaLaunchKernelEx(&config, join_kernel<T, kDim, kTiles>, p);
        if (joined != cudaSuccess) return joined;
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
    return f.parts ? meta_bytes(f) + sizeof(float) * 2 * f.blocks * f.part_rows * (f.dim + 2) : 0;
}

template <class T>
cudaError_t launch_tree_attention(const TreeAttention &t, cudaStream_t s)
{
    const Attention &a = t.a;
    const TreePlan f = tree_plan(a);
    TreeParams p;
    p.t = t;
    p.pack = f.pack, p.nodes_per = f.nodes_per, p.packs = f.packs, p.pairs = f.pairs, p.part_rows = f.part_rows;
    if (!f.blocks) return cudaErrorInvalidValue;
    p.units = f.packs * f.pairs;
    p.least = f.parts ? kLeastPart : kWhole;
    p.by_pack = Divider(f.pack), p.by_pairs = Divider(f.pairs), p.by_group = Divider(a.group), p.by_blocks = Divider(f.blocks);
    p.meta = f.parts ? static_cast<int4 *>(a.workspace) : nullptr;
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
