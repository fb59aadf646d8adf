// drafts.cu -- drafted tokens after the model has run (include/rng.h): their
// verification against the target's probabilities, and the move of the accepted
// ones' cache rows.
//
// Verification.  A cluster of blocks has a batch entry, each block a slice of the
// vocabulary, each warp a run of the slice.  What the walk needs of the drafts
// (their probabilities at their parents) is fetched by one block for all at once,
// so that walking down accepted drafts reads shared memory only; in every block one
// warp walks, from the same numbers.  A row is read when a draft has been rejected:
// all warps sum what is left, max(p - c q, 0), and the blocks share their sums.  c
// only grows, so that what later rejections of the same row can leave is what the
// first one left: while there are more children to try, those tokens' p and q are
// kept in shared memory, as far as there is room, and later sums read little else.  The last token is looked
// for within the one run where the sum passes u[0] of the whole.
//
// The sums decide whole numbers, so they are kept in pairs of f32 (48 bits): f64
// would be slower than HBM here (2 operations a cycle and SM), and f32 sums would
// pick a neighbouring token about once in a thousand draws of a large vocabulary.
//
// What bounds it, measured: latency. One request of 32768 tokens: 8.5 us in a graph (the
// launch, then 1.3 us for what the walk needs, 2.2 for the walk, 0.9 for the row's sums, 3
// for the blocks' exchange and the token); each further rejection of the same row 3 us.
// 128 requests of 131072 tokens, 16 nodes (1.9 sums a request, 8 at most): 74 us for the
// 117 MB that are read; issue slots 37 %, and the last requests alone for a quarter of
// the time. Chosen drafts, 64 requests of 24 nodes: 23 us for 34 MB.
#include <cooperative_groups.h>

#include "attention.h"

namespace cg = cooperative_groups;

namespace rngk {
namespace {

constexpr int kMaxNodes = RNG_MAX_TREE_NODES;
constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxCluster = 8;
// Tokens that a warp keeps: 70 KB a block, three blocks an SM (four blocks with 800: 128 requests of 131072 tokens, mean
// of eight seeds, 87 us for 74).  Without draft probabilities four (22 us for 32 with three; six, which spill, 29).
constexpr int kMostKept = 1120;

struct VerifyParams {
    int32_t batch, nodes, vocab;
    const void *target, *draft;
    int64_t target_batch, target_node, draft_batch, draft_node;
    const int32_t *tokens, *parents;
    const float *uniforms;
    uint32_t key, first;
    int32_t *path, *accepted, *out;
    int32_t run;   // tokens of a warp, a multiple of 32
    int32_t room;  // of which so many have room in shared memory
};

// A number or a sum as a pair of f32, error-free additions (Knuth's two-sum) and
// products with intrinsics, which the compiler leaves as they are.
struct Pair {
    float hi, lo;
    __device__ __forceinline__ void add(float x)
    {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
        hi = s;
    }
    __device__ __forceinline__ void add(const Pair &x)
    {
        add(x.hi);
        lo = __fadd_rn(lo, x.lo);
    }
    // As large a first number as there is (it is the larger of the two already).
    __device__ __forceinline__ Pair normal() const
    {
        const float s = __fadd_rn(hi, lo);
        return Pair{s, __fsub_rn(lo, __fsub_rn(s, hi))};
    }
};

__device__ __forceinline__ Pair times(float a, float b)
{
    const float t = __fmul_rn(a, b);
    return Pair{t, __fmaf_rn(a, b, -t)};
}
__device__ __forceinline__ Pair times(const Pair &a, const Pair &b)
{
    Pair t = times(a.hi, b.hi);
    t.lo = __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, t.lo));
    return t.normal();
}
__device__ __forceinline__ Pair plus(Pair a, const Pair &b)
{
    a.add(b);
    return a.normal();
}
__device__ __forceinline__ Pair minus(const Pair &a, const Pair &b) { return plus(a, Pair{-b.hi, -b.lo}); }
__device__ __forceinline__ bool less(const Pair &a, const Pair &b)  // of normal pairs
{
    return __fadd_rn(__fsub_rn(a.hi, b.hi), __fsub_rn(a.lo, b.lo)) < 0.0f;
}

// max(p - c q, 0): the product's error by a fused multiply-add, the difference's by
// two-sum.
__device__ __forceinline__ Pair left_of(float p, float q, const Pair &c)
{
    const float t = __fmul_rn(c.hi, q), te = __fmaf_rn(c.hi, q, -t);
    const float s = __fsub_rn(p, t), b = __fsub_rn(s, p);
    const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(s, b)), __fadd_rn(t, b));
    const float lo = __fsub_rn(__fsub_rn(e, te), __fmul_rn(c.lo, q));
    const float hi = __fadd_rn(s, lo);
    const bool some = hi > 0.0f;  // (not for NaN)
    return Pair{some ? hi : 0.0f, some ? __fsub_rn(lo, __fsub_rn(hi, s)) : 0.0f};
}

// Two sums at a time.
struct Pairs {
    float2 hi, lo;
    __device__ __forceinline__ static float2 sub(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }
    __device__ __forceinline__ void add(float2 x)
    {
        const float2 s = add2(hi, x), b = sub(s, hi);
        lo = add2(lo, add2(sub(hi, sub(s, b)), sub(x, b)));
        hi = s;
    }
    // p - q, of p at or above 0 and q taken down to p: the difference's error as in a fast two-sum.
    __device__ __forceinline__ void add_left(float2 p, float2 q)
    {
        p = make_float2(fmaxf(p.x, 0.0f), fmaxf(p.y, 0.0f)), q = make_float2(fminf(q.x, p.x), fminf(q.y, p.y));
        const float2 s = sub(p, q);
        add(s);
        lo = add2(lo, sub(sub(p, s), q));
    }
};

// What the walk needs, the same in every block of a cluster.
struct Nodes {
    int32_t parent[kMaxNodes], token[kMaxNodes];
    float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];  // probabilities at the parent's row
    int32_t stands[kMaxNodes];                       // as its parent's first child to be tried
};

// What a block's warps do next.
struct Command {
    enum Kind : int32_t { kEnd, kSum, kSumKept, kFind } kind;
    int32_t node;
    Pair c;
    bool removed;        // whether bits are set
    bool keeps;          // kSum: whether tokens that have something left are kept
    int32_t begin, end, stood;  // kFind: the run, and where its token goes
};

__device__ __forceinline__ Pair shuffled_up(const Pair &a, int d)
{
    return Pair{__shfl_up_sync(0xFFFFFFFFu, a.hi, d), __shfl_up_sync(0xFFFFFFFFu, a.lo, d)};
}
__device__ __forceinline__ Pair from_lane(const Pair &a, int l)
{
    return Pair{__shfl_sync(0xFFFFFFFFu, a.hi, l), __shfl_sync(0xFFFFFFFFu, a.lo, l)};
}
// The sum of the first kCount (a power of two) lanes' values, in all of those.
template <int kCount>
__device__ __forceinline__ Pair over_lanes(Pair sum)
{
#pragma unroll
    for (int d = kCount / 2; d; d /= 2)
        sum = plus(sum, Pair{__shfl_xor_sync(0xFFFFFFFFu, sum.hi, d), __shfl_xor_sync(0xFFFFFFFFu, sum.lo, d)});
    return sum;
}

// Looks for the first of some parts for which the sum up to it exceeds the bar, or,
// where rounding leaves none, for the last with any weight.
struct Search {
    Pair bar, before;
    // Among the first kCount lanes' parts; before becomes the sum before the one found.
    template <int kCount>
    __device__ __forceinline__ int32_t pick(const Pair &w, int32_t lane)
    {
        Pair up_to = w;
#pragma unroll
        for (int d = 1; d < kCount; d *= 2) {
            const Pair y = shuffled_up(up_to, d);
            if (lane >= d) up_to = plus(up_to, y);
        }
        const bool any_weight = w.hi > 0.0f && lane < kCount;
        const uint32_t any = __ballot_sync(0xFFFFFFFFu, any_weight), over = __ballot_sync(0xFFFFFFFFu, any_weight && less(bar, plus(before, up_to)));
        if (!over) bar = Pair{INFINITY, 0.0f};  // and so on from here
        const int32_t found = over ? __ffs(over) - 1 : any ? 31 - __clz(any) : 0;
        before = plus(before, from_lane(minus(up_to, w), found));
        return found;
    }
};

template <class T, bool kDraft>
__global__ void __launch_bounds__(kThreads, kDraft ? 3 : 4) verify_kernel(const __grid_constant__ VerifyParams v)
{
    // without draft probabilities, a bit to a token of the block's slice; with them, the kept tokens' p and q
    extern __shared__ uint32_t dynamic[];
    uint32_t *removed = dynamic;
    float2 *kept = reinterpret_cast<float2 *>(dynamic) + threadIdx.x / 32 * v.room;
    __shared__ Nodes n;
    __shared__ Pair totals[2][kMaxCluster];
    __shared__ Pair sums[kWarps];
    __shared__ int32_t counts[kWarps], resumes[kWarps], path[kMaxNodes];  // a warp's kept tokens, and from where on none are
    __shared__ Command command;
    __shared__ Search search;
    const cg::cluster_group cluster = cg::this_cluster();
    const int32_t rank = static_cast<int32_t>(cluster.block_rank()), blocks = static_cast<int32_t>(cluster.num_blocks());
    const int32_t entry = static_cast<int32_t>(blockIdx.x) / blocks, x = threadIdx.x, warp = x / 32, lane = x % 32;
    const T *target = static_cast<const T *>(v.target) + entry * v.target_batch;
    const T *draft = static_cast<const T *>(v.draft) + entry * v.draft_batch;
    const int64_t at0 = static_cast<int64_t>(entry) * v.nodes;

    // A block's shared memory is written by the cluster's first only when all of its blocks are known to run: they say so
    // here, and the first waits for it when its loads have been issued.
    cluster.barrier_arrive();
    int32_t parent = -2, token = -1;
    float u = 0.0f, p = 0.0f, q = 1.0f;
    if (rank == 0) {
        if (x < v.nodes) {
            parent = x == 0 ? -1 : v.parents ? v.parents[at0 + x] : x - 1, token = v.tokens[at0 + x];
            u = v.uniforms ? v.uniforms[at0 + x] : lowbias32::uniform_of(draw32(v.key, v.first + static_cast<uint32_t>(at0) + x));
            if (parent < 0 || parent >= x || token < 0 || token >= v.vocab) {
                parent = -2;  // never stands
            } else {
                p = to_f32(target[parent * v.target_node + token]);
                if (kDraft) q = to_f32(draft[parent * v.draft_node + token]);
            }
        }
    }
    cluster.barrier_wait();
    if (rank == 0 && x < kMaxNodes) {
        for (int32_t r = 0; r < blocks; ++r) {
            Nodes &to = *cluster.map_shared_rank(&n, r);
            to.stands[x] = parent >= 0 && p > 0.0f && less(times(u, q).normal(), Pair{p, 0.0f});
            to.parent[x] = parent, to.token[x] = token, to.u[x] = u, to.p[x] = p, to.q[x] = q;
        }
    }
    const int32_t slice = v.run * kWarps, slice0 = rank * slice;
    if (!kDraft)
        for (int32_t w = x; w < slice / 32; w += kThreads) removed[w] = 0;
    cluster.sync();

    // ---- the walk's state, in the first warp of each block
    const int32_t words = (v.nodes + 31) / 32;
    int32_t at = 0, stood = 0;
    Pair c{0.0f, 0.0f}, mass{1.0f, 0.0f};
    int32_t tried = 0;               // children of `at` up to this node were tried
    bool known = true;               // whether mass is the present w's
    bool has_kept = false;           // whether the present row's tokens are in shared memory
    bool some_removed = false, ending = false, from_p = false;
    uint32_t parity = 0;
    auto next_child = [&] {
        for (int32_t k = tried / 32; k < words; ++k) {
            const int32_t j = 32 * k + lane;
            const uint32_t kids = __ballot_sync(0xFFFFFFFFu, j > tried && j < v.nodes && n.parent[j] == at);
            if (kids) return 32 * k + __ffs(kids) - 1;
        }
        return -1;
    };
    // Bits of the children of `at` that were rejected, in the block's slice.
    auto forget = [&] {
        for (int32_t j = lane; j < v.nodes; j += 32) {
            const uint32_t place = n.token[j] - slice0;
            if (n.parent[j] == at && place < static_cast<uint32_t>(slice)) removed[place / 32] = 0;
        }
        __syncwarp();
        some_removed = false;
    };
    if (x == 0) path[0] = 0;
    Command next{Command::kSum, 0, c, false, false, 0, 0, 0};

    for (;;) {
        if (warp == 0) {
            while (next.kind == Command::kSum && !ending) {
                const int32_t i = next_child();
                ending = i < 0;
                next.keeps = kDraft && !ending;
                if (ending || (kDraft && !known)) break;
                bool stands = n.stands[i] != 0;
                const int32_t t = n.token[i];
                Pair w = kDraft ? left_of(n.p[i], n.q[i], c) : Pair{fmaxf(n.p[i], 0.0f), 0.0f};
                if (tried > at) {  // not the first
                    bool again = false;
                    if (!kDraft)  // a token that was rejected once has nothing left
                        for (int32_t j = lane; j < i; j += 32) again = again || (n.parent[j] == at && n.token[j] == t);
                    if (__any_sync(0xFFFFFFFFu, again)) w.hi = 0.0f;
                    stands = w.hi > 0.0f && less(times(times(n.u[i], n.q[i]).normal(), mass), w);
                }
                if (stands) {
                    if (!kDraft && some_removed) forget();
                    at = tried = i, c = Pair{0.0f, 0.0f}, mass = Pair{1.0f, 0.0f};
                    known = true, has_kept = false;
                    ++stood;
                    if (lane == 0) path[stood] = i;
                    continue;
                }
                tried = i;
                if (kDraft) {
                    c.add(mass), c = c.normal(), known = false;
                } else {
                    mass.add(-w.hi), mass = mass.normal();
                    const uint32_t place = t - slice0;
                    if (lane == 0 && place < static_cast<uint32_t>(slice)) removed[place / 32] |= 1u << place % 32;
                    some_removed = true;
                    __syncwarp();
                }
            }
            if (next.kind == Command::kSum && has_kept) next.kind = Command::kSumKept;
            next.node = at, next.c = c, next.removed = some_removed;
            if (lane == 0) command = next;
        }
        __syncthreads();
        const Command now = command;
        if (now.kind == Command::kEnd) break;
        const T *p = target + now.node * v.target_node, *q = draft + now.node * v.draft_node;
        // Without a rejection at this node c is 0, and the draft's row has no say, whatever it holds.
        const bool reads_q = kDraft && now.c.hi != 0.0f;
        // What is left of a token.
        auto left_at = [&](int32_t t, float a, float b) {
            if (kDraft) return reads_q ? left_of(a, b, now.c) : Pair{fmaxf(a, 0.0f), 0.0f};
            const uint32_t place = t - slice0;
            return Pair{a > 0.0f && !(now.removed && (removed[place / 32] >> place % 32 & 1u)) ? a : 0.0f, 0.0f};
        };
        auto fetch = [&](int32_t t) { return left_at(t, to_f32(p[t]), reads_q ? to_f32(q[t]) : 0.0f); };

        if (now.kind == Command::kFind) {
            // ---- the last token, in a run that all threads share: some adjacent tokens each
            const int32_t each = (now.end - now.begin + kThreads - 1) / kThreads;
            const int32_t from = min(now.begin + x * each, now.end), to = min(from + each, now.end);
            Pair mine{0.0f, 0.0f};
#pragma unroll 4
            for (int32_t t = from; t < to; ++t) mine.add(fetch(t));
            mine = mine.normal();
            const Pair sum = over_lanes<32>(mine);
            if (lane == 0) sums[warp] = sum;
            __syncthreads();
            Search s = search;
            if (s.pick<kWarps>(sums[lane % kWarps], lane) != warp) break;
            if (s.pick<32>(mine, lane) != lane) break;
            int32_t token = -1;
            for (int32_t t = from; t < to; ++t) {
                const Pair w = fetch(t);
                if (!(w.hi > 0.0f)) continue;
                token = t, s.before = plus(s.before, w);
                if (less(s.bar, s.before)) break;
            }
            v.out[at0 + now.stood] = token;
            break;
        }

        // ---- the sum of what is left of the row; a warp's part stays in `sums`, a block's in `totals`
        Pair sum{0.0f, 0.0f};
        const int32_t end = min(slice0 + (warp + 1) * v.run, v.vocab);
        int32_t begin = slice0 + warp * v.run;
        if (kDraft && now.kind == Command::kSumKept) {
            const int32_t count = counts[warp];
            constexpr int kAtOnce = 4;  // as many chains of additions
            Pair four[kAtOnce] = {};
            for (int32_t j = lane; j < count; j += 32 * kAtOnce) {
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const float2 pq = j + 32 * k < count ? kept[j + 32 * k] : make_float2(0.0f, 0.0f);
                    four[k].add(left_of(pq.x, pq.y, now.c));
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) sum.add(four[k]);
            begin = resumes[warp];
        }
        {
            constexpr int kAtOnce = kDraft ? 8 : 16;
            Pairs two{make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            // after one rejection c is 1, and without any 0: no product
            const bool plain = kDraft ? now.c.lo == 0.0f && (now.c.hi == 0.0f || now.c.hi == 1.0f) : !now.removed;
            int32_t count = 0, resume = end;
            bool keeps = kDraft && now.keeps && now.kind == Command::kSum;
            auto room_for = [&](int32_t t, int32_t tokens) {  // from t - lane on
                if (count + tokens <= v.room) return;
                keeps = false, resume = t - lane;
            };
            auto keep = [&](float a, float b) {
                const bool more = a > b;
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, more);
                if (more) kept[count + __popc(who & ((1u << lane) - 1u))] = make_float2(a, b);
                count += __popc(who);
            };
            int32_t t = begin + lane;
            for (; t - lane + 32 * kAtOnce <= end; t += 32 * kAtOnce) {
                float a[kAtOnce], b[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) a[k] = to_f32(p[t + 32 * k]), b[k] = reads_q ? to_f32(q[t + 32 * k]) : 0.0f;
                if (plain) {
#pragma unroll
                    for (int k = 0; k < kAtOnce; k += 2) two.add_left(make_float2(a[k], a[k + 1]), make_float2(b[k], b[k + 1]));
                } else {
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) sum.add(left_at(t + 32 * k, a[k], b[k]));
                }
                if (keeps) room_for(t, 32 * kAtOnce);
                if (keeps) {
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) keep(a[k], b[k]);
                }
            }
            for (; t - lane < end; t += 32) {
                const float a = t < end ? to_f32(p[t]) : 0.0f, b = reads_q && t < end ? to_f32(q[t]) : 0.0f;
                if (t < end) sum.add(left_at(t, a, b));
                if (keeps) room_for(t, 32);
                if (keeps) keep(a, b);
            }
            sum.add(Pair{two.hi.x, two.lo.x}), sum.add(Pair{two.hi.y, two.lo.y});
            if (kDraft && now.kind == Command::kSum && lane == 0) counts[warp] = count, resumes[warp] = resume;
        }
        sum = over_lanes<32>(sum.normal());
        if (lane == 0) sums[warp] = sum;
        __syncthreads();
        parity ^= 1u;
        if (warp == 0) {
            const Pair block = over_lanes<kWarps>(sums[lane % kWarps]);
            if (lane < blocks) *cluster.map_shared_rank(&totals[parity][rank], lane) = block;
        }
        cluster.sync();
        if (warp != 0) continue;
        const Pair part = lane < blocks ? totals[parity][lane] : Pair{0.0f, 0.0f};
        mass = from_lane(over_lanes<kMaxCluster>(part), 0), known = true;
        has_kept = now.kind == Command::kSumKept || now.keeps;
        next.kind = Command::kSum;
        if (!ending) continue;
        if (!(mass.hi > 0.0f) && !from_p) {  // nothing is left: from p itself
            from_p = true, c = Pair{0.0f, 0.0f}, has_kept = false;
            if (!kDraft) forget();
            continue;
        }
        // ---- the walk's end
        int32_t *out = v.out + at0, *out_path = v.path + at0;
        if (rank == 0) {
            if (lane == 0) v.accepted[entry] = stood;
            for (int32_t k = lane; k < v.nodes; k += 32) {
                out_path[k] = k <= stood ? path[k] : -1;
                if (k != stood) out[k] = k < stood ? n.token[path[k + 1]] : -1;
            }
        }
        next.kind = Command::kEnd;
        if (!(mass.hi > 0.0f)) {
            if (rank == 0 && lane == 0) out[stood] = -1;
            continue;
        }
        Search s{times(Pair{n.u[0], 0.0f}, mass), Pair{0.0f, 0.0f}};
        if (s.pick<kMaxCluster>(part, lane) != rank) continue;
        const int32_t run = s.pick<kWarps>(sums[lane % kWarps], lane);
        next.kind = Command::kFind, next.begin = slice0 + run * v.run, next.end = min(next.begin + v.run, v.vocab), next.stood = stood;
        if (lane == 0) search = s;
    }
}

// ---- the accepted rows' move

constexpr int kKeepThreads = 256, kCachesAtOnce = 128, kRowsAtOnce = 8;

struct KeepParams {
    uint4 *cache[kCachesAtOnce];
    int32_t batch, nodes, len_k, vectors, head_vectors, chunks, blocks;  // 16-byte vectors of a row and of a head
    int64_t stride_batch, stride_row, stride_head;                       // in vectors
    const int32_t *lengths, *path, *accepted;
    int32_t *new_lengths;
};

__device__ __forceinline__ int32_t within(int32_t v, int32_t most) { return min(max(v, 0), most); }

// A thread moves one vector of every row, kRowsAtOnce rows' loads at a time: row
// path[k] > k is read before a later step may write it, since path ascends.  The
// blocks after the caches' write the new lengths.  Bound by latency (the path, then
// the rows): 64 caches of 32 entries, 8 heads of 128, 3.4 rows an entry: 24 MB in 7 us.
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepParams p)
{
    const int32_t room = p.len_k - p.nodes;
    if (static_cast<int32_t>(blockIdx.x) >= p.blocks) {
        const int32_t b = (blockIdx.x - p.blocks) * kKeepThreads + threadIdx.x;
        if (b < p.batch) p.new_lengths[b] = (p.lengths ? within(p.lengths[b], room) : room) + within(p.accepted[b], p.nodes - 1) + 1;
        return;
    }
    const int32_t chunk = blockIdx.x % p.chunks, rest = blockIdx.x / p.chunks, b = rest % p.batch;
    const int32_t at = chunk * kKeepThreads + threadIdx.x;
    if (at >= p.vectors) return;
    const int32_t kept = within(p.accepted[b], p.nodes - 1), cached = p.lengths ? within(p.lengths[b], room) : room;
    const int32_t *path = p.path + static_cast<int64_t>(b) * p.nodes;
    uint4 *row = p.cache[rest / p.batch] + b * p.stride_batch + cached * p.stride_row + at / p.head_vectors * p.stride_head +
                 at % p.head_vectors;
    for (int32_t k0 = 1; k0 <= kept; k0 += kRowsAtOnce) {
        uint4 value[kRowsAtOnce];
        bool moves[kRowsAtOnce];
#pragma unroll
        for (int32_t r = 0; r < kRowsAtOnce; ++r) {
            const int32_t from = k0 + r <= kept ? path[k0 + r] : 0;
            moves[r] = from > k0 + r && from < p.nodes;
            if (moves[r]) value[r] = row[from * p.stride_row];
        }
#pragma unroll
        for (int32_t r = 0; r < kRowsAtOnce; ++r)
            if (moves[r]) row[(k0 + r) * p.stride_row] = value[r];
    }
}

}  // namespace

cudaError_t launch_cache_keep(const CacheKeep &c, void *const *caches, int32_t count, cudaStream_t s)
{
    KeepParams p;
    p.batch = c.batch, p.nodes = c.nodes, p.len_k = c.len_k;
    p.head_vectors = c.dim / 8;
    p.stride_batch = c.strides.batch / 8, p.stride_row = c.strides.len / 8, p.stride_head = c.strides.head / 8;
    p.lengths = c.lengths, p.path = c.path, p.accepted = c.accepted, p.new_lengths = c.new_lengths;
    if (static_cast<int64_t>(c.heads) * p.head_vectors > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.vectors = c.heads * p.head_vectors;
    p.chunks = (p.vectors + kKeepThreads - 1) / kKeepThreads;
    const int64_t each = static_cast<int64_t>(p.chunks) * c.batch, lengths = c.new_lengths ? (c.batch + kKeepThreads - 1) / kKeepThreads : 0;
    if (each * kCachesAtOnce + lengths > 0x7FFFFFFF) return cudaErrorInvalidValue;
    for (int32_t at = 0; at == 0 || at < count; at += kCachesAtOnce) {
        const int32_t some = count - at < kCachesAtOnce ? count - at : kCachesAtOnce;
        for (int32_t i = 0; i < some; ++i) p.cache[i] = static_cast<uint4 *>(caches[at + i]);
        p.blocks = static_cast<int32_t>(each * some);
        const unsigned blocks = static_cast<unsigned>(p.blocks + (at == 0 ? lengths : 0));
        if (blocks == 0) continue;
        keep_kernel<<<blocks, kKeepThreads, 0, s>>>(p);
        note_launch();
    }
    return cudaGetLastError();
}

namespace {

// ---- argument checks

struct Range {
    const char *name;
    const void *p;
    uint64_t bytes;
    size_t element;
    bool output, optional;
};

template <size_t N>
rng_status check_ranges(const char *what, const Range (&r)[N])
{
    for (size_t i = 0; i < N; ++i) {
        if (!r[i].p) {
            if (!r[i].optional) return fail(RNG_EINVAL, "%s: %s is NULL", what, r[i].name);
            continue;
        }
        const uintptr_t at = reinterpret_cast<uintptr_t>(r[i].p);
        if (at % r[i].element) return fail(RNG_EINVAL, "%s: %s is not aligned to its %zu-byte element", what, r[i].name, r[i].element);
        if (r[i].bytes > UINTPTR_MAX - at) return fail(RNG_EINVAL, "%s: %s runs past the end of the address space", what, r[i].name);
        for (size_t j = 0; j < i; ++j) {
            const uintptr_t other = reinterpret_cast<uintptr_t>(r[j].p);
            if (r[j].p && (r[i].output || r[j].output) && at < other + r[j].bytes && other < at + r[i].bytes)
                return fail(RNG_EINVAL, "%s: %s and %s overlap", what, r[j].name, r[i].name);
        }
    }
    return RNG_OK;
}

// Bytes from a [batch, nodes, vocab] array's address to its end; false for a stride that it cannot have.
bool extent(const int64_t (&stride)[2], const rng_verify_drafts_args &a, size_t size, uint64_t *bytes)
{
    const double most = static_cast<double>(a.batch - 1) * stride[0] + static_cast<double>(a.nodes - 1) * stride[1] + a.vocab;
    if (stride[0] < 0 || stride[1] < 0 || most * size > static_cast<double>(INT64_MAX)) return false;
    *bytes = size * (static_cast<uint64_t>(a.batch - 1) * stride[0] + static_cast<uint64_t>(a.nodes - 1) * stride[1] + a.vocab);
    return true;
}

template <class T, bool kDraft>
cudaError_t launch_verify(const VerifyParams &v, int cluster, cudaStream_t s)
{
    const auto kernel = verify_kernel<T, kDraft>;
    static std::atomic<bool> done[16];
    cudaError_t e = allow_shared(kernel, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(static_cast<unsigned>(v.batch) * cluster);
    config.blockDim = dim3(kThreads);
    config.dynamicSmemBytes = kDraft ? v.room * kWarps * sizeof(float2) : v.run * kWarps / 8;
    config.stream = s;
    cudaLaunchAttribute shape;
    shape.id = cudaLaunchAttributeClusterDimension;
    shape.val.clusterDim.x = cluster, shape.val.clusterDim.y = shape.val.clusterDim.z = 1;
    config.attrs = &shape, config.numAttrs = 1;
    e = cudaLaunchKernelEx(&config, kernel, v);
    if (e != cudaSuccess) return e;
    note_launch();
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_verify(const VerifyParams &v, int cluster, cudaStream_t s)
{
    return v.draft ? launch_verify<T, true>(v, cluster, s) : launch_verify<T, false>(v, cluster, s);
}

}  // namespace
}  // namespace rngk

using namespace rngk;

extern "C" {

rng_status rng_verify_drafts(const rng_verify_drafts_args *args, void *stream)
{
    static const char what[] = "rng_verify_drafts";
    if (!args) return fail(RNG_EINVAL, "%s: args is NULL", what);
    const rng_verify_drafts_args &a = *args;
    if (a.dtype != RNG_F32 && a.dtype != RNG_F16 && a.dtype != RNG_BF16)
        return fail(RNG_EINVAL, "%s: unknown dtype %d", what, a.dtype);
    if (a.batch < 0 || a.batch > 1 << 24) return fail(RNG_EINVAL, "%s: batch = %d is outside 0 .. 2^24", what, a.batch);
    if (a.nodes < 1 || a.nodes > RNG_MAX_TREE_NODES)
        return fail(RNG_EINVAL, "%s: nodes = %d is outside 1 .. %d", what, a.nodes, RNG_MAX_TREE_NODES);
    if (a.vocab < 1 || a.vocab > 1 << 23) return fail(RNG_EINVAL, "%s: vocab = %d is outside 1 .. 2^23", what, a.vocab);
    if (a.batch == 0) return RNG_OK;
    const size_t size = a.dtype == RNG_F32 ? 4 : 2;
    const uint64_t flat = uint64_t(4) * a.batch * a.nodes;
    uint64_t target = 0, draft = 0;
    if (!extent(a.target_stride, a, size, &target) || (a.draft && !extent(a.draft_stride, a, size, &draft)))
        return fail(RNG_EINVAL, "%s: a stride is negative or too large", what);
    const Range ranges[] = {{"target", a.target, target, size, false, false},
                            {"draft", a.draft, draft, size, false, true},
                            {"tokens", a.tokens, flat, 4, false, false},
                            {"parents", a.parents, flat, 4, false, true},
                            {"uniforms", a.uniforms, flat, 4, false, true},
                            {"path", a.path, flat, 4, true, false},
                            {"accepted", a.accepted, uint64_t(4) * a.batch, 4, true, false},
                            {"out_tokens", a.out_tokens, flat, 4, true, false}};
    if (rng_status st = check_ranges(what, ranges)) return st;
    VerifyParams v{a.batch, a.nodes, a.vocab, a.target, a.draft, a.target_stride[0], a.target_stride[1], a.draft_stride[0],
                   a.draft_stride[1], a.tokens, a.parents, a.uniforms, seed_key(a.seed), a.first_counter, a.path, a.accepted,
                   a.out_tokens, 0, 0};
    // More blocks to a request while each keeps 2048 tokens and the SMs hold all of them (about three each); past that only
    // where a block has so much to read that the next ones' wait is made up for, and more where already some wait.  Nine
    // nodes, drawn (chosen), f32, clusters of 1, 2, 4, 8, us: 16 x 8192 13, 11, 10, 11 (10, 9, 10, 9); 16 x 131072 108, 58,
    // 31, 20 (57, 32, 19, 14); 128 x 8192 16, 14, 17, 27 (10, 9, 11, 18); 128 x 32768 32, 24, 22, 28 (19, 14, 13, 19); 128 x
    // 131072 140, 86, 57, 54 (65, 41, 27, 31); 256 x 8192 17, 19, 25, 47 (11, 11, 20, 31); 256 x 16384 24, 22, 28, 43 (14, 13,
    // 19, 35); 256 x 65536 91, 57, 54, 69 (41, 28, 31, 41).
    const int64_t room = 3 * static_cast<int64_t>(sm_count());
    int cluster = 1;
    for (; cluster < kMaxCluster; cluster *= 2) {
        const int64_t now = static_cast<int64_t>(a.batch) * cluster;
        const int32_t least = 2 * now <= room ? 2048 : now <= room ? 12288 : a.draft ? 24576 : 49152;
        if (a.vocab <= cluster * least) break;
    }
    const int32_t warps = cluster * kWarps;
    v.run = ((a.vocab + warps - 1) / warps + 31) / 32 * 32;
    v.room = v.run < kMostKept ? v.run : kMostKept;
    clear_error();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a.dtype == RNG_F32   ? launch_verify<float>(v, cluster, s)
                          : a.dtype == RNG_F16 ? launch_verify<__half>(v, cluster, s)
                                               : launch_verify<__nv_bfloat16>(v, cluster, s);
    return e == cudaSuccess ? RNG_OK : cuda_fail(e, what);
}

}  // extern "C"
