// attention_fwd.cu -- attention forward (include/rng.h, rng_attention_fwd) on
// the tensor cores.
//
// A block works on two "slots" of 128 query rows by 128 keys.  For a slot's key
// tile, S = Q K^T goes to TMEM; the slot's threads take the rows of S,
// update the row's running maximum and sum, and write P = exp(S - max)
// back over S in 16 bits; O += P V accumulates in TMEM with P as the TMEM
// operand.  Two threads share a row, 64 keys each, so that four warps a
// scheduler hide each other's latencies; they agree on the row's maximum only
// when one of them has to raise it.  One thread issues all products, one warp
// the TMA loads of the key and value tiles, and while a slot's threads work on
// its scores the tensor core works for the other slot.
//   kSplitKeys = false: the slots are two tiles of queries that share the key
//     and value tiles (halving their traffic from L2);
//   kSplitKeys = true: one tile of queries, the slots take every other key
//     tile and are joined at the end.  For few rows, where the key axis is also
//     split over blocks, and joined by join_kernel.
// The query heads of one key head are `pack` adjacent rows of a tile, so that
// they read its keys once.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since its
// last rescaling: P then stays below 2^8, which 16 bits hold as well as 1.
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace rngk {
namespace {

constexpr int kTile = 128;          // rows of a slot, keys of a tile
constexpr int kHalf = kTile / 2;    // keys of a thread
// 2 x 256 for the slots, then a TMA warp, an MMA warp, two that only fill the warpgroup
constexpr int kThreads = 640;
constexpr uint32_t kTmaWarp = 16, kMmaWarp = 17;
// registers: 640 threads start with 96 each; 4 x 104 + 64 = 5 x 96
constexpr int kSlotRegisters = 104, kOtherRegisters = 64;
constexpr uint32_t kBox = 16384;    // bytes of 128 rows of 64 elements
constexpr float kLog2e = 1.4426950408889634f;

struct FwdParams {
    CUtensorMap q, k, v;
    Attention a;
    int32_t pack, units, q_tiles, splits, split_tiles;
    float *part;  // [splits][rows][dim padded + 2]: O, max, sum
};

template <int kDim, bool kSplitKeys>
struct Shape {
    static constexpr int kBoxes = kDim / 64;
    static constexpr int kQTiles = kSplitKeys ? 1 : 2;
    static constexpr int kStages = kDim == 64 ? 8 : kSplitKeys ? 5 : 4;
    static constexpr uint32_t kStageBytes = kBoxes * kBox;
    static constexpr uint32_t kRing = kQTiles * kStageBytes;  // where the ring begins
    static constexpr uint32_t kTable = kRing + kStages * kStageBytes;
};

// Barriers of a slot's 256 threads; slot_any also tells whether any of them
// asked.
__device__ __forceinline__ void slot_sync(int slot) { asm volatile("bar.sync %0, 256;" ::"r"(2 + slot) : "memory"); }
__device__ __forceinline__ bool slot_any(int slot, bool ask)
{
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 256, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(yes)
        : "r"(static_cast<uint32_t>(ask)), "r"(2 + slot)
        : "memory");
    return yes != 0;
}

template <class T, int kDim, bool kSplitKeys, bool kDrop, bool kBias>
__global__ void __launch_bounds__(kThreads, 1) attention_fwd_kernel(const __grid_constant__ FwdParams p)
{
    using S = Shape<kDim, kSplitKeys>;
    extern __shared__ uint8_t dynamic[];
    __shared__ alignas(8) uint64_t bars[2 * S::kStages + 8];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t stalled;
    __shared__ float tops[2][2][2][kTile], sums[2][2][kTile];  // [turn's parity][slot][half][row], [slot][half][row]
    const Attention &a = p.a;
    const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
    uint8_t *smem = dynamic + ((1024u - (smem_address(dynamic) & 1023u)) & 1023u);
    const uint32_t base = smem_address(smem);
    float *table = reinterpret_cast<float *>(smem + S::kTable);

    // ---- the block's work
    uint32_t x = blockIdx.x;
    const int32_t split = x % p.splits;
    x /= p.splits;
    int32_t unit, q_tile;
    if (a.causal) {  // the longest first
        unit = x % p.units, q_tile = p.q_tiles - 1 - x / p.units;
    } else {
        q_tile = x % p.q_tiles, unit = x / p.q_tiles;
    }
    const int32_t packs = a.heads / p.pack, b = unit / packs, pack = unit % packs;
    const int32_t head0 = pack * p.pack, head_kv = head0 / a.group;
    const int32_t rows_per = kTile / p.pack;  // positions of a tile
    const int32_t i0 = q_tile * S::kQTiles * rows_per;
    const int32_t keys = keys_of(a, b), pos0 = first_position(a, keys);
    // key tiles of each slot (both slots' are the block's when the keys are split)
    int32_t tile0 = split * p.split_tiles, count[2];
    for (int s = 0; s < 2; ++s) {
        const int32_t last = min(i0 + (kSplitKeys ? 1 : s + 1) * rows_per, a.len_q) - 1;  // the slot's last query
        int32_t end = a.causal ? min(keys, pos0 + last + 1) : keys;
        if (!kSplitKeys && i0 + s * rows_per >= a.len_q) end = 0;
        end = max(0, min((end + kTile - 1) / kTile - tile0, p.split_tiles));
        count[s] = end;
    }
    const int32_t tiles = max(count[0], count[1]);

    // ---- barriers, TMEM
    const uint32_t bar0 = smem_address(bars);
    const uint32_t full = bar0, empty = bar0 + 8 * S::kStages, scored = empty + 8 * S::kStages, ready = scored + 16,
                   done = ready + 16, q_full = done + 8, tail = q_full + 8;
    if (threadIdx.x == 0) {
        stalled = 0;
        for (int s = 0; s < S::kStages; ++s) barrier_init(full + 8 * s, 1), barrier_init(empty + 8 * s, 1);
        for (int s = 0; s < 2; ++s) barrier_init(scored + 8 * s, 1), barrier_init(ready + 8 * s, 8);
        barrier_init(done, 1), barrier_init(q_full, 1), barrier_init(tail, 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc<512>(smem_address(&tmem_base));
    if (kBias) {  // the bias by relative position, head head0 (pack is 1)
        const int32_t reach = bias_reach(a.buckets);
        for (int32_t t = threadIdx.x; t < 2 * reach; t += kThreads)
            table[t] = to_f32(static_cast<const T *>(a.table)[bucket_of(a.buckets, t - reach) * a.heads + head0]);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base;
    if (warp >= kTmaWarp) {
      give_registers<kOtherRegisters>();
      if (warp == kTmaWarp) {
        // ---- TMA: the queries, then K_0 .. K_{lead-1} and alternately V_n, K_{n+lead}
        constexpr int kLead = kSplitKeys ? 2 : 1;
        const bool one = elect_one();
        if (one && tiles) {
            prefetch_map(&p.k), prefetch_map(&p.v);
            barrier_expect(q_full, S::kQTiles * S::kStageBytes);
            for (int t = 0; t < S::kQTiles; ++t)
                for (int c = 0; c < S::kBoxes; ++c)
                    tma_load_5d(base + t * S::kStageBytes + c * kBox, &p.q, q_full, c * 64, 0, i0 + t * rows_per, pack, b);
        }
        uint32_t use = 0;
        auto load = [&](const CUtensorMap *map, int32_t n, bool values) {
            const uint32_t stage = use % S::kStages, dst = base + S::kRing + stage * S::kStageBytes;
            const uint32_t bar = full + 8 * stage;
            barrier_wait(empty + 8 * stage, (use / S::kStages & 1u) ^ 1u, &stalled);
            const int32_t j0 = (tile0 + n) * kTile;
            // keys past n(b) that the array holds: whatever they are, P's zeros must meet zeros
            const bool past = values && j0 + kTile > keys && keys < a.len_k;
            const uint32_t on = past ? tail : bar;
            if (one) {
                barrier_expect(on, S::kStageBytes);
                for (int c = 0; c < S::kBoxes; ++c) tma_load_5d(dst + c * kBox, map, on, c * 64, 0, j0, head_kv, b);
            }
            if (past) {
                barrier_wait(tail, 0, &stalled);
                uint8_t *rows = smem + S::kRing + stage * S::kStageBytes;
                for (int c = 0; c < S::kBoxes; ++c)
                    for (uint32_t o = max(0, keys - j0) * 128u + lane * 16u; o < kBox; o += 512u)
                        *reinterpret_cast<uint4 *>(rows + c * kBox + o) = make_uint4(0, 0, 0, 0);
                fence_async_shared();
                __syncwarp();
                if (one) barrier_arrive(bar);
            }
            ++use;
        };
        for (int32_t n = 0; n < kLead && n < tiles; ++n) load(&p.k, n, false);
        for (int32_t n = 0; n < tiles; ++n) {
            load(&p.v, n, true);
            if (n + kLead < tiles) load(&p.k, n + kLead, false);
        }
        if (stalled && one)  // nothing may land after the block has ended
            for (uint32_t u = use > S::kStages ? use - S::kStages : 0; u < use; ++u)
                for (uint32_t tries = 0; tries < 100000 && !barrier_try(full + 8 * (u % S::kStages), u / S::kStages & 1u); ++tries) {}
      } else if (warp == kMmaWarp) {
        // ---- MMA
        if (elect_one() && tiles) {
            constexpr uint32_t kScores = mma_shape<T>(kTile, false), kOut = mma_shape<T>(kDim, true);
            uint32_t use = 0, given0 = 0, given1 = 0;
            auto acquire = [&] {
                const uint32_t stage = use % S::kStages;
                barrier_wait(full + 8 * stage, use / S::kStages & 1u, &stalled);
                tmem_fence_after();
                return stage;
            };
            auto release = [&] {
                mma_commit(empty + 8 * (use % S::kStages));
                ++use;
            };
            auto scores = [&](int slot, uint32_t stage) {
                const uint32_t q = base + (kSplitKeys ? 0 : slot) * S::kStageBytes, k = base + S::kRing + stage * S::kStageBytes;
                const uint64_t qd = row_major_tile(q), kd = row_major_tile(k);
#pragma unroll
                for (int i = 0; i < kDim / 16; ++i) {
                    constexpr uint32_t kStep = 16;  // descriptors count 16 bytes
                    const uint32_t o = (i / 4 * kBox + i % 4 * 32) / kStep;
                    mma_step(tmem + slot * 256, qd + o, kd + o, kScores, i > 0);
                }
                mma_commit(scored + 8 * slot);
            };
            auto products = [&](int slot, uint32_t stage, bool first) {
                const uint32_t v = base + S::kRing + stage * S::kStageBytes;
                barrier_wait(ready + 8 * slot, (slot ? given1++ : given0++) & 1u, &stalled);
                tmem_fence_after();
                const uint64_t vd = column_major_tile(v, S::kBoxes > 1 ? kBox : 1024);
#pragma unroll
                for (int i = 0; i < kTile / 16; ++i)
                    mma_step_tmem(tmem + slot * 256 + kTile, tmem + slot * 256 + i / 4 * kHalf + i % 4 * 8, vd + i * (2048 / 16), kOut,
                                  !first || i > 0);
            };
            barrier_wait(q_full, 0, &stalled);
            if (kSplitKeys) {
#pragma unroll 1
                for (int32_t n = -2; n < tiles; ++n) {
                    if (n >= 0) products(n & 1, acquire(), n < 2), release();
                    if (n + 2 < tiles) scores(n & 1, acquire()), release();
                }
            } else {
                // the stages of V_n and K_{n+1}, each released when both slots have used it
#pragma unroll 1
                for (int32_t n = -1; n < tiles; ++n) {
                    const uint32_t vs = n >= 0 ? acquire() : 0;
                    uint32_t ks = S::kStages;
#pragma unroll 1
                    for (int s = 0; s < 2; ++s) {
                        if (n >= 0 && n < count[s]) products(s, vs, n == 0);
                        if (n + 1 < count[s]) {
                            if (ks == S::kStages) {
                                if (n >= 0) ++use;
                                ks = acquire();
                                if (n >= 0) --use;
                            }
                            scores(s, ks);
                        }
                    }
                    if (n >= 0) release();
                    if (n + 1 < tiles) release();
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
        const uint32_t mine = tmem + slot * 256 + lanes + half * kHalf;              // the thread's scores, then its P
        const uint32_t out = tmem + slot * 256 + lanes + kTile + half * (kDim / 2);  // its half of O's columns
        const int32_t row0 = (kSplitKeys ? 0 : slot * kTile);
        const int32_t warp_i = i0 + (row0 + (warp % 4) * 32) / p.pack;  // the warp's first query
        const int32_t i = i0 + (row0 + r) / p.pack, head = head0 + r % p.pack, pos = pos0 + i;
        const bool valid = i < a.len_q, any = warp_i < a.len_q;
        const int64_t index = (static_cast<int64_t>(b) * a.heads + head) * a.len_q + i;
        const uint32_t counter = a.first + static_cast<uint32_t>(index) * static_cast<uint32_t>(a.len_k) + half * kHalf;
        const int32_t visible = a.causal ? min(keys, pos + 1) : keys;
        const int32_t warp_visible = a.causal ? min(keys, pos0 + warp_i + 1) : keys;  // the least of the warp's
        const bool plain = !kBias && a.scale > 0.0f;
        // scores are held before (plain) or after their scaling and bias; base two is for the exponential
        const float to_base2 = plain ? a.scale * kLog2e : kLog2e, to_natural = plain ? a.scale : 1.0f;
        const int32_t reach = kBias ? bias_reach(a.buckets) : 0;
        const float bias_low = kBias ? table[0] : 0.0f, bias_high = kBias ? table[2 * reach - 1] : 0.0f;
        float top = -INFINITY, sum = 0.0f;
        uint32_t turn = 0;
        for (int32_t n = kSplitKeys ? slot : 0; n < count[kSplitKeys ? 0 : slot]; n += kSplitKeys ? 2 : 1, ++turn) {
            const int32_t j0 = (tile0 + n) * kTile + half * kHalf;
            barrier_wait(scored + 8 * slot, turn & 1u, &stalled);
            tmem_fence_after();
            uint32_t s[2][32];
            float tile_top = -INFINITY;
            if (any) {
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_load32(s[c], mine + 32 * c);
                tmem_wait_load(s);
                if (kBias) {
                    // relative positions of the warp's pairs: beyond the last bucket's start on one side, or by the table
                    const int32_t low = j0 - (pos0 + warp_i + 31), high = j0 + kHalf - 1 - (pos0 + warp_i);
                    const float2 scale = make_float2(a.scale, a.scale);
                    if (high <= -a.buckets.max_distance || low >= a.buckets.max_distance) {
                        const float v = high < 0 ? bias_low : bias_high;
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
                } else if (!plain) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[c][e] = __float_as_uint(__uint_as_float(s[c][e]) * a.scale);
                }
                if (j0 + kHalf > warp_visible) {
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
                tile_top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
            }
            // A new maximum, and O and the sums brought to it: at the first finite score, or 2^8 above the old one.
            // Where one of the slot's threads needs it, its rows' halves meet.
            const bool want = tile_top > top && (top == -INFINITY || (tile_top - top) * to_base2 > 8.0f);
            if (slot_any(slot, want)) {
                float(&meet)[2][kTile] = tops[turn & 1u][slot];
                meet[half][r] = tile_top;
                slot_sync(slot);
                const float most = fmaxf(meet[0][r], meet[1][r]);
                const bool raise = most > top && (top == -INFINITY || (most - top) * to_base2 > 8.0f);
                if (any && __any_sync(0xFFFFFFFFu, raise)) {
                    const float next = raise ? most : top;
                    const float fade = raise ? exp2_approx((top - next) * to_base2) : 1.0f;
                    sum *= fade;
                    top = next;
                    if (turn) {
#pragma unroll 1
                        for (int c = 0; c < kDim / 32; ++c) {
                            uint32_t o[16];
                            tmem_load16(o, out + 16 * c);
                            tmem_wait_load16(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fade);
                            tmem_store16(out + 16 * c, o);
                        }
                    }
                }
            }
            if (any) {
                // exp2((s - top) to_base2): as one multiply-add, or, where a bias may be the type's
                // lowest value, with the difference taken first
                const float from = top == -INFINITY ? 0.0f : -top, shift = from * to_base2;
                const float2 from2 = make_float2(from, from), shift2 = make_float2(shift, shift);
                const float2 base2 = make_float2(to_base2, to_base2);
                float2 total = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 v = make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                        const float2 f = plain ? fma2(v, base2, shift2) : mul2(add2(v, from2), base2);
                        const float2 q = make_float2(exp2_approx(f.x), exp2_approx(f.y));
                        total = add2(total, q);
                        s[c][e] = __float_as_uint(q.x), s[c][e + 1] = __float_as_uint(q.y);
                    }
                    if (kDrop) drop32(a.mask, counter + (tile0 + n) * kTile + 32 * c, s[c]);
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        w[e / 2] = pack2<T>(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                    tmem_store16(mine + 16 * c, w);
                }
                sum += total.x + total.y;
                tmem_wait_store();
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) barrier_arrive(ready + 8 * slot);
        }

        // ---- the result
        if (tiles) {
            barrier_wait(done, 0, &stalled);
            tmem_fence_after();
        }
        sums[slot][half][r] = sum;
        if (kSplitKeys && half == 0) tops[0][slot][0][r] = top;
        float *hand = reinterpret_cast<float *>(smem + S::kRing);  // the ring, which nothing reads any more
        const bool two = kSplitKeys && tiles > 1;
        if (two && slot == 1 && any) {  // slot 1 hands its part to slot 0
#pragma unroll
            for (int c = 0; c < kDim / 64; ++c) {
                uint32_t o[1][32];
                tmem_load32(o[0], out + 32 * c);
                tmem_wait_load(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) hand[(half * (kDim / 2) + 32 * c + e) * kTile + r] = __uint_as_float(o[0][e]);
            }
        }
        asm volatile("bar.sync 1, 512;" ::: "memory");
        if (any && (!kSplitKeys || slot == 0)) {
            float weight = 1.0f, other = 0.0f;
            sum = sums[slot][0][r] + sums[slot][1][r];
            if (two) {
                const float top1 = tops[0][1][0][r], sum1 = sums[1][0][r] + sums[1][1][r], most = fmaxf(top, top1);
                weight = top == -INFINITY ? 0.0f : exp2_approx((top - most) * to_base2);
                other = top1 == -INFINITY ? 0.0f : exp2_approx((top1 - most) * to_base2);
                sum = sum * weight + sum1 * other;
                top = most;
            }
            const bool whole = p.splits == 1;
            float *part = p.part + (static_cast<int64_t>(split) * a.batch * a.heads * a.len_q + index) * (kDim + 2);
            const float scale = !whole ? 1.0f : sum == 0.0f ? 0.0f : a.mask.scale / sum;
            T *o_row = static_cast<T *>(a.out) + b * a.os.batch + i * a.os.len + head * a.os.head;
#pragma unroll
            for (int c = 0; c < kDim / 64; ++c) {
                uint32_t o[1][32] = {};
                const int col = half * (kDim / 2) + 32 * c;
                if (tiles) {
                    tmem_load32(o[0], out + 32 * c);
                    tmem_wait_load(o);
                }
                if (valid) {
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        v[e] = __uint_as_float(o[0][e]);
                        if (two) v[e] = v[e] * weight + hand[(col + e) * kTile + r] * other;
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
            if (valid && half == 0) {
                if (!whole)
                    part[kDim] = top * to_natural, part[kDim + 1] = sum;
                else if (a.lse)
                    a.lse[index] = sum == 0.0f ? -INFINITY : top * to_natural + logf(sum);
            }
        }
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) tmem_free<512>(tmem);
}

// Joins the key axis's splits: a warp to a row.
template <class T, int kDim>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ FwdParams p)
{
    const Attention &a = p.a;
    const int64_t rows = static_cast<int64_t>(a.batch) * a.heads * a.len_q;
    const int64_t index = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.y;
    if (index >= rows) return;
    const uint32_t lane = threadIdx.x;
    constexpr int kEach = kDim / 32;
    float top = -INFINITY, sum = 0.0f, o[kEach] = {};
    for (int32_t s = 0; s < p.splits; ++s) {
        const float *part = p.part + (s * rows + index) * (kDim + 2);
        const float t = part[kDim], l = part[kDim + 1];
        if (l == 0.0f) continue;  // saw nothing
        const float next = fmaxf(top, t), fade = exp2_approx((top - next) * kLog2e);
        const float weight = exp2_approx((t - next) * kLog2e);
        sum = sum * fade + l * weight;
        top = next;
#pragma unroll
        for (int k = 0; k < kEach; ++k) o[k] = o[k] * fade + part[lane * kEach + k] * weight;
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
    const int32_t rows_per = kTile / f.pack, tiles = (a.len_q + rows_per - 1) / rows_per;
    const int32_t key_tiles = (a.len_k + kTile - 1) / kTile;
    f.split_keys = tiles == 1;
    f.q_tiles = f.split_keys ? 1 : (tiles + 1) / 2;
    f.splits = 1, f.split_tiles = key_tiles < 1 ? 1 : key_tiles;
    if (f.split_keys && key_tiles > 2) {
        // about four blocks to an SM, of two key tiles or more
        const int64_t want = (4ll * sm_count() + f.units - 1) / f.units;
        const int64_t most = (key_tiles + 1) / 2;
        const int64_t splits = want < most ? want : most;
        f.split_tiles = static_cast<int32_t>((key_tiles + splits - 1) / splits);
        f.splits = (key_tiles + f.split_tiles - 1) / f.split_tiles;
    }
    return f;
}

template <class T, int kDim, bool kSplitKeys, bool kDrop, bool kBias>
cudaError_t launch(const FwdParams &p, cudaStream_t s)
{
    using S = Shape<kDim, kSplitKeys>;
    const auto kernel = attention_fwd_kernel<T, kDim, kSplitKeys, kDrop, kBias>;
    const size_t bytes = 1024 + S::kTable + (kBias ? 2 * bias_reach(p.a.buckets) * sizeof(float) : 0);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
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

template <class T, int kDim, bool kSplitKeys>
cudaError_t launch(const FwdParams &p, cudaStream_t s)
{
    const bool drop = p.a.mask.threshold != 0, bias = p.a.table != nullptr;
    if (drop) return bias ? launch<T, kDim, kSplitKeys, true, true>(p, s) : launch<T, kDim, kSplitKeys, true, false>(p, s);
    return bias ? launch<T, kDim, kSplitKeys, false, true>(p, s) : launch<T, kDim, kSplitKeys, false, false>(p, s);
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
    p.part = static_cast<float *>(a.workspace);
    if (static_cast<int64_t>(f.units) * f.q_tiles * f.splits > 0x7FFFFFFF) return cudaErrorInvalidValue;
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    cudaError_t e = make_heads_map(&p.q, bf16, a.q, a.qs, a.batch, a.len_q, a.heads, a.dim, f.pack, kTile);
    if (a.len_k > 0) {
        if (e == cudaSuccess) e = make_heads_map(&p.k, bf16, a.k, a.ks, a.batch, a.len_k, a.heads_kv, a.dim, 1, kTile);
        if (e == cudaSuccess) e = make_heads_map(&p.v, bf16, a.v, a.vs, a.batch, a.len_k, a.heads_kv, a.dim, 1, kTile);
    } else {
        p.k = p.v = p.q;  // not read
    }
    if (e != cudaSuccess) return e;
    if (f.dim == 64) return f.split_keys ? launch<T, 64, true>(p, s) : launch<T, 64, false>(p, s);
    return f.split_keys ? launch<T, 128, true>(p, s) : launch<T, 128, false>(p, s);
}

template cudaError_t launch_attention_fwd<__half>(const Attention &, cudaStream_t);
template cudaError_t launch_attention_fwd<__nv_bfloat16>(const Attention &, cudaStream_t);

}  // namespace rngk
