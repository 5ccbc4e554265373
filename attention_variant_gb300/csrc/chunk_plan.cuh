// chunk_plan.cuh -- how the work of a ragged chunk call is cut up
// (fwd_chunk.cu): the planning kernel, and what both attention paths share.
//
// Two lists: row blocks (entries of one or two blocks of TQ = 128 / G tokens)
// and few rows (requests whose tokens times G are at most kFewRows).  An
// entry's items are its KV heads -- pairs of KV heads on the few-row list,
// the last of an odd number by itself -- and an item's tiles its key tiles
// (times heads).  A list is one long line of tiles with a cost each; it is cut
// into equal parts, one a CTA; each list has a kernel, and the SMs are shared
// between the two by cost.
#pragma once

#include "common.cuh"
#include "fl_attn.h"
#include "launch.h"

namespace fl {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsSoftmax = 200;
constexpr uint32_t kRegsOther = 104;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther == kThreads * kRegsLaunch,
              "register split must equal the launch allocation");
constexpr int kInfo = 4; // items published ahead of the slowest role

__device__ uint32_t g_lib_error_word;

__device__ __forceinline__ uint32_t bar(const uint64_t &b) { return ptx::smem_u32(&b); }

__device__ __forceinline__ WaitCtl wait_ctl(const ChunkParams &p, uint32_t *abort_flag)
{
    WaitCtl wc;
    wc.abort_flag = abort_flag;
    wc.timeout_cycles = p.timeout_ns * 21 / 10; // 2.1 cycles per ns at the maximum clock
    wc.err_user = p.err_user;
    wc.err_lib = &g_lib_error_word;
    return wc;
}

// Keys [lo, hi) that the tokens at positions first .. last see.  (first may be far
// below 0, before the sequence, and the window as long as an int goes.)
__device__ __forceinline__ void key_range(const ChunkParams &p, int L, int first, int last, int &lo, int &hi)
{
    lo = p.window ? max(0, max(first, 0) - p.window + 1) : 0;
    hi = p.causal ? min(L, last + 1) : L;
}

__device__ __forceinline__ bool is_few(const ChunkParams &p, int n_tok) { return n_tok * p.G <= kFewRows; }

// a / b for a >= 0, b > 0: costs are 64-bit, but their division is only where it has to be.
__device__ __noinline__ int64_t div64(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0)
        return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// KV heads of an entry's items (the last may have fewer).
__device__ __forceinline__ int item_heads(const ChunkParams &p, const ChunkEntry &en)
{
    return is_few(p, en.n_tok) && p.Hk > 1 ? 2 : 1;
}

// Cost of an item with its full number of heads; an odd head's is less, but
// it comes last in its entry, so positions divide by this.
__device__ __forceinline__ int64_t item_cost(const ChunkParams &p, const ChunkEntry &en)
{
    return static_cast<int64_t>(en.n_tiles) * item_heads(p, en) * en.tile_cost +
           (is_few(p, en.n_tok) ? p.cost_few_item : p.cost_item);
}

__device__ __forceinline__ int64_t entry_cost(const ChunkParams &p, const ChunkEntry &en)
{
    const int heads = item_heads(p, en);
    return static_cast<int64_t>(en.n_tiles) * p.Hk * en.tile_cost +
           static_cast<int64_t>(heads == 2 ? (p.Hk + 1) >> 1 : p.Hk) *
               (is_few(p, en.n_tok) ? p.cost_few_item : p.cost_item);
}

// What the planning kernel wrote, read past L1: a second kernel may have
// started before it (below).
template <class T>
__device__ __forceinline__ T load_plan(const T *src)
{
    static_assert(sizeof(T) % 16 == 0, "16-byte words");
    union {
        T value;
        uint4 word[sizeof(T) / 16];
    } u;
#pragma unroll
    for (size_t i = 0; i < sizeof(T) / 16; ++i)
        u.word[i] = __ldcg(reinterpret_cast<const uint4 *>(src) + i);
    return u.value;
}

// The kernels of the two paths.  The first one's CTAs start beside the planning
// kernel: they set up and then wait for the plan.  The second one is launched
// when every CTA of the first has seen the plan.  That it sees it, too, follows
// from a word that a thread of the first releases and all of its own acquire;
// should it not come soon, they wait for the first kernel's end.  (The release is
// a softmax thread's, which has nothing to do yet: from the producer it cost 1 us.)
// Its CTAs take the SMs as those without work leave them.  Both end with a
// wait for the one before: the second stands for the first to what follows, and
// a CTA of the first that gave up early is not gone before the plan is there.
// (One kernel for both: the path laid out second started 6 to 9 us late, its
// instructions fetched from memory.)

// A CTA's place among its kernel's parts.  CTAs go to SMs in order, two by two,
// but for the first one, whose neighbour is the SM that the planning kernel
// still held; it gets the last, so that the two SMs of a pair run one path: the
// instructions of both do not fit what they share (a pair that ran both took
// 20% longer).  Where CTAs are placed otherwise the results are the same.
__device__ __forceinline__ int part_of(const ChunkParams &p)
{
    const int c = blockIdx.x;
    return p.second ? c : c + 1 == p.n_cta ? 0 : c + 1;
}

// At the start: a CTA of the second kernel without work (kind 0: row blocks, 1:
// few rows) has only to wait for the first.
__device__ __forceinline__ bool idle_second(const ChunkParams &p, int kind, int part)
{
    if (!p.second)
        return false;
    ptx::launch_dependents();
    int tries = 32; // 20 us
    while (ptx::load_acquire(p.seen) != p.seen_mark && --tries)
        ;
    if (!tries)
        ptx::wait_dependency();
    if (__ldcg(&p.parts[kind * p.n_cta + part].parts))
        return false;
    ptx::wait_dependency();
    return true;
}

// The word of the first kernel for the second.  The softmax warps.
__device__ __forceinline__ void tell_second(const ChunkParams &p, int part)
{
    if (!p.second && p.seen_mark && part == 0 && threadIdx.x == kThreads - 1) {
        ptx::wait_dependency();
        ptx::store_release(p.seen, p.seen_mark);
    }
    __syncwarp();
}

// The CTA's part, which begins at tile k of item h of entry e.  A warp.
__device__ __forceinline__ void read_part(const ChunkParams &p, int kind, int part, ChunkPart &me, int &e, int &h,
                                          int &k)
{
    if (!p.second) {
        ptx::wait_dependency();
        ptx::launch_dependents();
    }
    me = load_plan(p.parts + kind * p.n_cta + part);
    e = me.entry;
    h = me.item;
    k = me.tile;
}

// Part c of `parts` covers the cost units x with c total / parts <= x <
// (c + 1) total / parts, and a tile belongs to the part of its first unit.
struct PartRange {
    int k_end;          // the part's tiles of the item: k .. k_end - 1
    int first, n_parts; // the item's first part and number of parts
};

__device__ __forceinline__ PartRange part_range(int64_t x0, int n_tiles, int tile_cost, int k, int64_t x_end,
                                                int64_t total, int part, int parts)
{
    PartRange r;
    r.k_end = static_cast<int>(min(static_cast<int64_t>(n_tiles), (x_end - x0 + tile_cost - 1) / tile_cost));
    r.first = k == 0 ? part : static_cast<int>(x0 * parts / total);
    const int last = r.k_end == n_tiles
                         ? part
                         : static_cast<int>((x0 + static_cast<int64_t>(n_tiles - 1) * tile_cost) * parts / total);
    r.n_parts = last - r.first + 1;
    return r;
}

// Layouts of an item's partial results (one buffer a slot):
//   JOIN_PAIR   the slot's own rows: [D columns][128 rows]
//   JOIN_HALF   one row block, the slot's half of the columns: [D / 2][128]
//               then, for both, m, l and the sum of the rounded P: [3][128]
//   JOIN_FEW    [16 rows][128 dimensions], m [16], then each warp's sums of l:
//               [4 warps][16]
enum : int { JOIN_PAIR = 0, JOIN_HALF = 1, JOIN_FEW = 2 };

// Floats of one slot's buffer, and the place of a slot's buffer of a CTA
// (buffer 1: the item begins in that CTA, 0: it began before).
template <int D>
__device__ __forceinline__ float *partial(const ChunkParams &p, int cta, int buf, int slot)
{
    return p.partials + (static_cast<int64_t>(cta * 2 + buf) * 2 + slot) * ((D + 4) * 128);
}

// ------------------------------------------------------------------ planning

constexpr int kPlanThreads = 1024;
constexpr int kPlanNear = 128; // entries of each list kept at hand

// What one scan of the planning kernel adds up: places on the two lists
// (16 bits each; at most kPlanThreads a round) and costs.
struct PlanSum {
    int places;
    int64_t cost[2];
};
__device__ __forceinline__ PlanSum operator+(const PlanSum &a, const PlanSum &b)
{
    return PlanSum{a.places + b.places, {a.cost[0] + b.cost[0], a.cost[1] + b.cost[1]}};
}
__device__ __forceinline__ int shfl_up(int x, int d) { return __shfl_up_sync(0xffffffffu, x, d); }
__device__ __forceinline__ PlanSum shfl_up(const PlanSum &x, int d)
{
    return PlanSum{__shfl_up_sync(0xffffffffu, x.places, d),
                   {__shfl_up_sync(0xffffffffu, x.cost[0], d), __shfl_up_sync(0xffffffffu, x.cost[1], d)}};
}

// Barrier of the planning kernel's first `threads` threads.
__device__ __forceinline__ void plan_sync(int threads)
{
    if (threads == 32)
        __syncwarp();
    else
        ptx::named_barrier_sync(1, threads);
}

// Inclusive sum over the first `threads` threads (a power of two of warps, at
// most 32); the total is left in s_warp[31].
template <class T>
__device__ __forceinline__ T block_scan(T x, T *s_warp, int threads)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = threads >> 5;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const T y = shfl_up(x, d);
        if (lane >= d)
            x = x + y;
    }
    plan_sync(threads); // the last scan's sums have been read
    if (warps == 1) {
        if (lane == 31)
            s_warp[31] = x;
        plan_sync(threads);
        return x;
    }
    if (lane == 31)
        s_warp[warp] = x;
    plan_sync(threads);
    if (warp == 0) {
        T w = lane < warps ? s_warp[lane] : T{};
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const T y = shfl_up(w, d);
            if (lane >= d)
                w = w + y;
        }
        s_warp[lane] = w;
    }
    plan_sync(threads);
    return warp ? s_warp[warp - 1] + x : x;
}

// What the planning kernel's threads share.
struct PlanShared {
    int scan[32];
    PlanSum sum[32];
    int ent[kPlanThreads + 1];                            // first entry of each request of the round
    int t0[kPlanThreads], n[kPlanThreads], len[kPlanThreads];
    int64_t cum[2][kPlanThreads];                         // cost before each of the first entries
    ChunkEntry entry[2][kPlanNear];                       // and the very first ones
    int most;                                             // cost of the dearest tile of a row block
    int count[2];                                         // entries and cost of the lists
    int64_t total[2];
};

// The lists of entries, by `threads` threads.
template <int D>
__device__ __forceinline__ void plan_entries(const ChunkParams &p, PlanShared &sm, int threads)
{
    const int tid = threadIdx.x;
    const int per = 2 * p.TQ; // tokens per entry
    int count[2] = {0, 0};
    int64_t cum[2] = {0, 0};
    uint32_t err = 0;
    if (tid == 0)
        sm.most = 0;
    for (int b0 = 0; b0 < p.batch; b0 += threads) {
        const int b = b0 + tid;
        int n = 0, t0 = 0, L = 0;
        if (b < p.batch) {
            t0 = __ldg(p.cu_q + b);
            int t1 = __ldg(p.cu_q + b + 1);
            L = __ldg(p.kv_lens + b);
            if (t0 < 0 || t1 > p.T || t1 < t0 || L < 0 || (L > p.max_kv && p.strict))
                err |= FL_DEVERR_LENGTHS;
            t0 = min(max(t0, 0), p.T);
            t1 = min(max(t1, t0), p.T);
            n = t1 - t0;
            L = min(max(L, 0), p.max_kv);
        }
        const int ent = fast_div(n + per - 1, p.div_per);
        const int end = block_scan(ent, sm.scan, threads);
        sm.ent[tid] = end - ent;
        if (tid == threads - 1)
            sm.ent[threads] = end;
        sm.t0[tid] = t0;
        sm.n[tid] = n;
        sm.len[tid] = L;
        plan_sync(threads);
        const int n_round = sm.ent[threads];
        for (int e0 = 0; e0 < n_round; e0 += threads) {
            const int e = e0 + tid;
            ChunkEntry en{};
            PlanSum add{};
            int kind = -1;
            if (e < n_round) {
                int lo = 0, hi = threads - 1; // the last request that starts at or before e
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (sm.ent[mid] <= e)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                const int at = (e - sm.ent[lo]) * per;
                en.b = b0 + lo;
                en.t0 = sm.t0[lo] + at;
                en.n_tok = min(per, sm.n[lo] - at);
                en.L = sm.len[lo];
                en.pos0 = en.L - sm.n[lo] + at;
                int k0, k1;
                key_range(p, en.L, en.pos0, en.pos0 + en.n_tok - 1, k0, k1);
                en.key_lo = k0;
                kind = is_few(p, en.n_tok) ? 1 : 0;
                const int tile = kind ? kFewTile : chunk_key_tile(D);
                en.lo = k0 / tile;
                en.n_tiles = max(1, (max(k1, 0) + tile - 1) / tile - en.lo);
                en.tile_cost = kind ? p.cost_few : en.n_tok > p.TQ ? p.cost_pair : p.cost_single;
                add.places = kind ? 1 << 16 : 1;
                const int64_t cost = entry_cost(p, en);
                add.cost[0] = kind ? 0 : cost;
                add.cost[1] = kind ? cost : 0;
                if (!kind)
                    atomicMax(&sm.most, en.tile_cost);
            }
            const PlanSum sum = block_scan(add, sm.sum, threads);
            if (kind >= 0) {
                const int at = (kind ? count[1] + (sum.places >> 16) : count[0] + (sum.places & 0xffff)) - 1;
                en.cum = kind ? cum[1] + sum.cost[1] - add.cost[1] : cum[0] + sum.cost[0] - add.cost[0];
                // overlapping requests may give more than fit: those are dropped
                if (at < p.max_entries) {
                    p.entries[kind * p.max_entries + at] = en;
                    if (at < kPlanThreads)
                        sm.cum[kind][at] = en.cum;
                    if (at < kPlanNear)
                        sm.entry[kind][at] = en;
                }
            }
            count[0] += sm.sum[31].places & 0xffff;
            count[1] += sm.sum[31].places >> 16;
            cum[0] += sm.sum[31].cost[0];
            cum[1] += sm.sum[31].cost[1];
        }
        plan_sync(threads); // the next round overwrites the requests
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
        if (count[kind] > p.max_entries) {
            err |= FL_DEVERR_LENGTHS;
            count[kind] = p.max_entries;
            const ChunkEntry &last = p.entries[(kind + 1) * p.max_entries - 1];
            cum[kind] = last.cum + entry_cost(p, last);
        }
    if (err && p.err_user)
        atomicOr(p.err_user, err);
    if (tid < 2) {
        sm.count[tid] = tid ? count[1] : count[0];
        sm.total[tid] = tid ? cum[1] : cum[0];
    }
}

// One block.  Its first `threads` threads list the entries (as few as make it
// one round: the barriers cost what they have to wait for), then all of them
// cut the parts, one a thread.
template <int D>
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkParams p, int threads)
{
    __shared__ PlanShared sm;
    ptx::launch_dependents();
    if (static_cast<int>(threadIdx.x) < threads)
        plan_entries<D>(p, sm, threads);
    __syncthreads();
    // parts of each list by its share of the cost, in pairs (see part_of); a part is
    // at least one tile long, so that every part between the first and the last
    // of an item holds one of its tiles
    const int64_t cum[2] = {sm.total[0], sm.total[1]};
    int parts[2];
    {
        const int64_t both = cum[0] + cum[1];
        int share = cum[0] ? p.n_cta : 0;
        if (cum[0] && cum[1])
            share = min(max(static_cast<int>(div64(cum[0] * p.n_cta + both, 2 * both)) * 2, 2), p.n_cta - 2);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const int64_t tile = kind ? p.cost_few : sm.most, least = max(tile, static_cast<int64_t>(p.cost_least));
            int g = kind ? p.n_cta - share : share;
            if (cum[kind] < least * g)
                g = static_cast<int>(div64(cum[kind] + least - 1, least));
            if (g > 1 && cum[kind] < tile * g)
                --g;
            parts[kind] = g;
        }
    }
    for (int c = threadIdx.x; c < 2 * p.n_cta; c += blockDim.x) {
        ChunkPart out{};
        const int kind = c >= p.n_cta ? 1 : 0, part = kind ? c - p.n_cta : c, g = kind ? parts[1] : parts[0];
        if (part < g) {
            const int64_t total = kind ? cum[1] : cum[0];
            const int64_t x = div64(total * part + g - 1, g);  // first cost unit of this part
            // the last entry that starts at or before x
            int lo = 0, hi = sm.count[kind] - 1;
            if (hi >= kPlanThreads) {
                const ChunkEntry *list = p.entries + kind * p.max_entries;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (list[mid].cum <= x)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
            }
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (sm.cum[kind][mid] <= x)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const ChunkEntry en = lo < kPlanNear ? sm.entry[kind][lo] : p.entries[kind * p.max_entries + lo];
            out.at = en;
            const int64_t cost = item_cost(p, en);
            out.total = total;
            out.end = div64(total * (part + 1) + g - 1, g);
            out.cta = (kind ? parts[0] : 0) + part;
            out.parts = g;
            out.n_entries = sm.count[kind];
            out.entry = lo;
            out.item = static_cast<int>(div64(x - en.cum, cost));
            const int64_t in = x - en.cum - out.item * cost;
            out.tile = static_cast<int>(div64(in + en.tile_cost - 1, en.tile_cost));
        }
        p.parts[c] = out;
        if (!kind)
            p.joins[part].n_parts = 0;
    }
}

// ------------------------------------------------------------------ joining
//
// Items whose keys were cut: O = sum 2^(m_q - M) O_q / sum 2^(m_q - M) l_q over
// the parts q, in their order.  A kernel of its own: joining inside the
// attention kernel (by the last CTA to come) put a fence, an atomic and three
// rounds of loads on one CTA's path, 5 to 8 us at the end of the step; here
// they are spread over 8 blocks an item.  The partials are not read by
// read-only loads, which may not see what a kernel writes that still runs when
// this one starts: row blocks, which use a line once, go past L1.

constexpr int kJoinThreads = 128, kJoinSplit = 4;

__device__ __forceinline__ void join_write(const ChunkParams &p, int64_t tok, int64_t head, int dim, float o, float l)
{
    p.out[tok * p.o_st + head * p.o_sh + dim] = __float2bfloat16(l == 0.f ? 0.f : o * ptx::rcp_approx(l));
}

__device__ __forceinline__ void join_lse(const ChunkParams &p, int64_t tok, int64_t head, float m, float l)
{
    if (p.lse)
        p.lse[head * p.l_sh + tok] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
}

// Row-block layouts: a row per thread, N / kJoinSplit columns.
template <int N, int D>
__device__ __forceinline__ void join_block(const ChunkParams &p, const ChunkJoin &jn, int cta, int slot, int z)
{
    constexpr int C = N / kJoinSplit;
    const int r = threadIdx.x, n_parts = jn.n_parts;
    if (r >= jn.rows[slot])
        return;
    float M = kNegInf, l = 0.f, lr = 0.f, o[C];
#pragma unroll
    for (int i = 0; i < C; ++i)
        o[i] = 0.f;
    const float *b0 = partial<D>(p, cta, 1, slot) + r;
#pragma unroll 4
    for (int q = 0; q < n_parts; ++q)
        M = fmaxf(M, __ldcg((q ? partial<D>(p, cta + q, 0, slot) + r : b0) + N * 128));
    const float M0 = M == kNegInf ? 0.f : M;
#pragma unroll 2
    for (int q = 0; q < n_parts; ++q) {
        const float *b = q ? partial<D>(p, cta + q, 0, slot) + r : b0;
        const float m = __ldcg(b + N * 128), w = ptx::ex2(m - M0);
        l = fmaf(w, __ldcg(b + (N + 1) * 128), l);
        lr = fmaf(w, __ldcg(b + (N + 2) * 128), lr);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            // the O of a part without a key of this row was not written
            const float v = __ldcg(b + (z * C + i) * 128);
            o[i] = m == kNegInf ? o[i] : fmaf(w, v, o[i]);
        }
    }
    const int r_tok = fast_div(r, p.div_g);
    const int64_t tok = jn.t0[slot] + r_tok, head = jn.kvh * p.G + r - r_tok * p.G;
    const float inv = lr == 0.f ? 0.f : ptx::rcp_approx(lr);
    const int col = (N < D ? slot * N : 0) + z * C;
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + tok * p.o_st + head * p.o_sh + col);
#pragma unroll
    for (int i = 0; i < C; i += 8)
        dst[i / 8] = make_uint4(ptx::pack_bf16(o[i] * inv, o[i + 1] * inv), ptx::pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                                ptx::pack_bf16(o[i + 4] * inv, o[i + 5] * inv),
                                ptx::pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
    if (z == 0 && (N == D || slot == 0))
        join_lse(p, tok, head, M, l);
}

// Few rows: a dimension per thread (at D = 64 half the threads a row), a part
// per lane while the weights are made.
template <int D>
__device__ __forceinline__ void join_few(const ChunkParams &p, const ChunkJoin &jn, int cta, int slot, int z)
{
    constexpr int R = kFewRows, kDepth = 16, kPerBlock = 128 / D;
    const int lane = threadIdx.x & 31, dim = threadIdx.x & (D - 1), n_parts = jn.n_parts;
    auto part = [&](int q) { return partial<D>(p, cta + q, q == 0 ? 1 : 0, slot); };
    for (int n = z * kPerBlock + static_cast<int>(threadIdx.x) / D; n < jn.rows[slot]; n += kJoinSplit * kPerBlock) {
        float M = kNegInf;
        for (int q = lane; q < n_parts; q += 32)
            M = fmaxf(M, part(q)[R * 128 + n]);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        const float M0 = M == kNegInf ? 0.f : M;
        float l = 0.f, o = 0.f;
        for (int q0 = 0; q0 < n_parts; q0 += 32) {
            float w = 0.f, a = 0.f;
            if (q0 + lane < n_parts) {
                const float *s = part(q0 + lane) + R * 128 + n;
                w = ptx::ex2(s[0] - M0);
#pragma unroll
                for (int k = 1; k <= 4; ++k)
                    a += s[R * k];
                a *= w;
            }
#pragma unroll
            for (int d = 16; d; d >>= 1)
                a += __shfl_xor_sync(0xffffffffu, a, d);
            l += a;
            for (int q = q0; q < min(q0 + 32, n_parts); q += kDepth) {
                float v[kDepth];
#pragma unroll
                for (int i = 0; i < kDepth; ++i)
                    v[i] = q + i < n_parts ? part(q + i)[n * 128 + dim] : 0.f;
#pragma unroll
                for (int i = 0; i < kDepth; ++i)
                    o = fmaf(__shfl_sync(0xffffffffu, w, (q + i) & 31), v[i], o);
            }
        }
        const int s = fast_div(n, p.div_g);
        const int64_t tok = jn.t0[slot] + s, head = (jn.kvh + slot) * p.G + n - s * p.G;
        join_write(p, tok, head, dim, o, l);
        if (dim == 0)
            join_lse(p, tok, head, M, l);
    }
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const __grid_constant__ ChunkParams p)
{
    ptx::wait_dependency();
    const int cta = blockIdx.x, slot = blockIdx.y, z = blockIdx.z;
    if (cta + slot + z == 0 && threadIdx.x == 0)
        *p.seen = 0; // a replay of this call has the same mark
    const ChunkJoin jn = p.joins[cta];
    if (jn.n_parts < 2)
        return;
    if (jn.mode == JOIN_FEW)
        join_few<D>(p, jn, cta, slot, z);
    else if (jn.mode == JOIN_PAIR)
        join_block<D, D>(p, jn, cta, slot, z);
    else
        join_block<D / 2, D>(p, jn, cta, slot, z);
}

} // namespace
} // namespace fl
