// fwd_chunk.cu -- attention of ragged chunks of new tokens over the cache
// that holds them (serving: prompts, parts of prompts and single tokens in
// one call), paged or contiguous; D = 64 or 128.
//
// Mathematics: the online softmax of softmax_tile.cuh; rows whose keys are
// split over several SMs leave partial (m, l, O) and are joined by
//     M = max m_i,  O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
//
// Work.  The query rows of a (request, KV head) are its tokens times the G
// query heads of the group, token by token: a block of TQ = 128 / G tokens
// fills the 128 rows of an MMA, so that even one token of a grouped head
// shares every key load among its heads.  An item is two such blocks (or the
// last one) of one request and KV head, against the key tiles any of its rows
// sees.  Lengths live on the device, so a one-block planning kernel lists the
// items' entries with a running sum of their cost, cuts the whole sum into
// equal parts and gives each CTA one: CTAs start and stop in the middle of an
// item's keys, wherever the cut falls, so a single long conversation spreads
// over the GPU as evenly as a full batch, and a batch needs no heuristics for
// the number of splits.  At most the first and last item of a CTA are shared;
// these leave partials in the workspace, and the last CTA to arrive (a ticket
// per warp of rows) joins them in the order of the keys.
//
// CTA (persistent, one per SM, 384 threads; the roles and the TMEM layout of
// the standard forward kernel, see fwd_standard.cu):
//   warp  0     walks the CTA's items, publishes each to the other roles,
//               loads Q (double-buffered across items) and the K/V tiles by TMA
//   warp  1     issues S = Q K^T for both slots; TMEM owner
//   warps 2, 3  issue O += P V for slot 0, slot 1
//   warps 4-11  two softmax warpgroups, one thread per row
// A slot is a 128-row softmax pipeline.  An item of two row blocks gives each
// slot a block, and they share every K/V tile (pair); an item of one block
// (single tokens, short chunks) gives both slots the same rows and every
// second key tile, and the slots' results are joined in the epilogue, each
// warpgroup reading both accumulators from TMEM for half of the columns.
// Warps that hold no row of the item skip the arithmetic.
//
// K/V tiles are 112 keys at D = 64 and 64 at D = 128 (TMEM budget of the
// standard kernel), loaded as boxes of 16 keys: the largest that divides the
// tile and every page size.  Keys no row may see never reach the sums: logits
// are replaced by -inf, and as 0 * NaN is not 0, the S warp zeroes those rows
// of V in shared memory (only in tiles at the ends of the cache or window).
#include <cuda_bf16.h>
#include <cstdint>

#include "common.cuh"
#include "fl_attn.h"
#include "launch.h"
#include "softmax_tile.cuh"

namespace fl {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsSoftmax = 200;
constexpr uint32_t kRegsOther = 104;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther == kThreads * kRegsLaunch,
              "register split must equal the launch allocation");
constexpr int kBox = 16; // keys per TMA box
constexpr int kInfo = 4; // items published ahead of the slowest role

template <int D>
struct ChunkCfg {
    static_assert(D == 64 || D == 128, "head dimension");
    static constexpr int kBN = chunk_key_tile(D);
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr bool kOnes = D <= 64; // sum of the rounded P from a ones column block
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kRowBytes = 128;
    static constexpr uint32_t kGroupBytes = 8 * kRowBytes;
    static constexpr uint32_t kQHalf = BM * kRowBytes;
    static constexpr uint32_t kKVHalf = kBN * kRowBytes;
    static constexpr uint32_t kTileBytes = kHalves * kQHalf;
    static constexpr uint32_t kKVBytes = kHalves * kKVHalf;
    static constexpr uint32_t kOnesBytes = kOnes ? kTileBytes : 16;
    static constexpr uint32_t kDvExt = kOnes ? D + 16 : D;
    static constexpr uint32_t kColSum = D;
    static constexpr uint32_t kColS = 0, kStrideS = kBN;
    static constexpr uint32_t kColO = 2 * kBN, kStrideO = kDvExt;
    static constexpr uint32_t kColP = 384, kStrideP = kBN / 2;
    static constexpr uint32_t kColX = kColP + 2 * kStrideP, kStrideX = 8; // the slots' (m, l, l_round)
    static_assert(kColO + 2 * kDvExt <= kColP && kColX + 2 * kStrideX <= 512, "TMEM budget");
    static_assert(kBN % kBox == 0 && kBN <= 128, "key tile");
};

// A CTA's part of an item, as the producer publishes it.
struct Item {
    int stop;
    int pair;                    // the slots hold two row blocks (else one, every second tile)
    int u_lo, u_hi;              // key tiles of this part
    int first[2], hi[2];         // slot's tiles: first, first + step, ... < hi
    int step;
    int t0[2], rows[2], pos0[2]; // slot's first token row, rows, first position
    int L, key_lo;               // cached keys; lowest key that any row of the item sees
    int kvh;
    int part, n_parts;           // first CTA of the item, number of CTAs
    int mine;                    // this part's buffer: 0 or 1
};

template <int D>
struct __align__(1024) ChunkSmem {
    using C = ChunkCfg<D>;
    uint8_t q[2][2][C::kTileBytes]; // [Q buffer][slot]
    uint8_t k[C::kStages][C::kKVBytes];
    uint8_t v[C::kStages][C::kKVBytes];
    uint8_t ones[C::kOnesBytes];
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[C::kStages], kv_empty[C::kStages];
    uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
    uint64_t turn[2];
    uint64_t x_full[2], x_free[2]; // join of the two slots (one row block)
    uint64_t final_bar[3];
    uint64_t info_full[kInfo], info_empty[kInfo];
    Item info[kInfo];
    uint32_t tmem_base;
    uint32_t abort_flag;
};

__device__ uint32_t g_lib_error_word;

template <int D>
struct KernelCtx {
    ChunkSmem<D> *sm;
    uint32_t tmem;
    WaitCtl wc;
};

__device__ __forceinline__ uint32_t bar(const uint64_t &b) { return ptx::smem_u32(&b); }

// Keys [lo, hi) that the tokens at positions first .. last see.
__device__ __forceinline__ void key_range(const ChunkParams &p, int L, int first, int last, int &lo, int &hi)
{
    lo = p.window ? max(0, first - p.window + 1) : 0;
    hi = p.causal ? min(L, last + 1) : L;
}

// ------------------------------------------------------------------ planning

constexpr int kPlanThreads = 1024;

template <class T>
__device__ __forceinline__ T block_scan(T x, T *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const T y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d)
            x += y;
    }
    __syncthreads(); // the last scan's sums have been read
    if (lane == 31)
        s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T w = s_warp[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const T y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d)
                w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    return x + (warp ? s_warp[warp - 1] : T(0));
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p)
{
    __shared__ int s_scan[32];
    __shared__ int64_t s_scan64[32];
    __shared__ int s_ent[kPlanThreads + 1]; // first entry of each request of the round
    __shared__ int s_t0[kPlanThreads], s_n[kPlanThreads], s_len[kPlanThreads];
    __shared__ int64_t s_cum[kPlanThreads]; // cost before each of the first entries
    __shared__ int s_wide;
    const int tid = threadIdx.x;
    const int per = 2 * p.TQ; // tokens per entry
    int n_entries = 0;
    int64_t cum = 0;
    uint32_t err = 0;
    for (int c = tid; c < 8 * p.n_cta; c += kPlanThreads)
        p.tickets[c] = 0;
    if (tid == 0)
        s_wide = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int n = 0, t0 = 0, L = 0;
        if (b < p.batch) {
            t0 = __ldg(p.cu_q + b);
            int t1 = __ldg(p.cu_q + b + 1);
            L = __ldg(p.kv_lens + b);
            if (t0 < 0 || t1 > p.T || t1 < t0)
                err |= FL_DEVERR_LENGTHS;
            t0 = min(max(t0, 0), p.T);
            t1 = min(max(t1, t0), p.T);
            n = t1 - t0;
            L = min(max(L, 0), p.max_kv);
        }
        const int ent = (n + per - 1) / per;
        const int end = block_scan(ent, s_scan);
        s_ent[tid] = end - ent;
        if (tid == kPlanThreads - 1)
            s_ent[kPlanThreads] = end;
        s_t0[tid] = t0;
        s_n[tid] = n;
        s_len[tid] = L;
        __syncthreads();
        const int n_round = s_ent[kPlanThreads];
        for (int e0 = 0; e0 < n_round; e0 += kPlanThreads) {
            const int e = e0 + tid;
            ChunkEntry en{};
            int64_t cost = 0;
            if (e < n_round) {
                int lo = 0, hi = kPlanThreads - 1; // the last request that starts at or before e
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (s_ent[mid] <= e)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                const int at = (e - s_ent[lo]) * per;
                en.b = b0 + lo;
                en.t0 = s_t0[lo] + at;
                en.n_tok = min(per, s_n[lo] - at);
                en.L = s_len[lo];
                en.pos0 = en.L - s_n[lo] + at;
                int k0, k1;
                key_range(p, en.L, en.pos0, en.pos0 + en.n_tok - 1, k0, k1);
                en.key_lo = k0;
                en.lo = k0 / p.key_tile;
                en.n_tiles = max(1, (max(k1, 0) + p.key_tile - 1) / p.key_tile - en.lo);
                en.tile_cost = en.n_tok > p.TQ ? p.cost_pair : p.cost_single;
                cost = (static_cast<int64_t>(en.n_tiles) * en.tile_cost + p.cost_item) * p.Hk;
                if (en.n_tok > p.TQ)
                    s_wide = 1; // every writer writes 1
            }
            const int64_t incl = block_scan(cost, s_scan64);
            en.cum = cum + incl - cost;
            const int at = n_entries + e;
            if (e < n_round && at < p.max_entries) {
                p.entries[at] = en;
                if (at < kPlanThreads)
                    s_cum[at] = en.cum;
            }
            cum += s_scan64[31];
        }
        n_entries += n_round;
        __syncthreads(); // the next round overwrites the requests
    }
    if (n_entries > p.max_entries) { // overlapping requests: drop what does not fit
        err |= FL_DEVERR_LENGTHS;
        n_entries = p.max_entries;
        const ChunkEntry &last = p.entries[n_entries - 1];
        cum = last.cum + (static_cast<int64_t>(last.n_tiles) * last.tile_cost + p.cost_item) * p.Hk;
    }
    if (err && p.err_user)
        atomicOr(p.err_user, err);
    // parts: each at least one tile long, so that every CTA between the first
    // and the last of an item holds one of its tiles
    const int64_t least = max(s_wide ? p.cost_pair : p.cost_single, p.cost_least);
    const int parts = static_cast<int>(min(static_cast<int64_t>(p.n_cta), (cum + least - 1) / least));
    const bool short_part = parts > 1 && cum / parts < (s_wide ? p.cost_pair : p.cost_single);
    const int g = short_part ? parts - 1 : parts;
    if (tid == 0) {
        p.head->total = cum;
        p.head->n_entries = n_entries;
        p.head->parts = g;
    }
    if (tid >= g)
        return;
    const int64_t x = (cum * tid + g - 1) / g; // first cost unit of this part
    int lo = 0, hi = n_entries - 1;            // the last entry that starts at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int64_t at = mid < kPlanThreads ? s_cum[mid] : p.entries[mid].cum;
        if (at <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    const ChunkEntry &en = p.entries[lo];
    const int64_t cost = static_cast<int64_t>(en.n_tiles) * en.tile_cost + p.cost_item;
    ChunkStart st;
    st.entry = lo;
    st.head = static_cast<int>((x - en.cum) / cost);
    const int64_t in = x - en.cum - st.head * cost;
    st.tile = static_cast<int>(min((in + en.tile_cost - 1) / en.tile_cost, static_cast<int64_t>(en.n_tiles)));
    st.pad = 0;
    p.starts[tid] = st;
}

// ------------------------------------------------------------------ producer

template <int D>
__device__ void producer_role(const KernelCtx<D> &cx, const ChunkParams &p, const CUtensorMap *tm_q,
                              const CUtensorMap *tm_k, const CUtensorMap *tm_v)
{
    using C = ChunkCfg<D>;
    constexpr int kBN = C::kBN, kStages = C::kStages, kBoxes = kBN / kBox;
    ChunkSmem<D> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    const int cta = blockIdx.x;
    uint32_t kv_count = 0, item_count = 0;
    bool ok = true;
    const int64_t total = p.head->total;
    const int parts = p.head->parts, n_entries = p.head->n_entries;
    int e = n_entries, h = 0, k = 0;
    int64_t x_end = 0;
    if (cta < parts) {
        const ChunkStart st = p.starts[cta];
        e = st.entry;
        h = st.head;
        k = st.tile;
        x_end = (total * (cta + 1) + parts - 1) / parts;
    }
    for (;;) {
        // ---- the next part
        Item it;
        it.stop = 1;
        ChunkEntry en{};
        int k_end = 0;
        while (e < n_entries) {
            en = p.entries[e];
            const int64_t cost = static_cast<int64_t>(en.n_tiles) * en.tile_cost + p.cost_item;
            const int64_t x0 = en.cum + h * cost;
            if (x0 + static_cast<int64_t>(k) * en.tile_cost >= x_end) {
                e = n_entries; // the cut falls before this tile
                break;
            }
            if (k < en.n_tiles) {
                k_end = static_cast<int>(
                    min(static_cast<int64_t>(en.n_tiles), (x_end - x0 + en.tile_cost - 1) / en.tile_cost));
                it.part = k == 0 ? cta : static_cast<int>(x0 * parts / total);
                const int last = k_end == en.n_tiles
                                     ? cta
                                     : static_cast<int>((x0 + static_cast<int64_t>(en.n_tiles - 1) * en.tile_cost) *
                                                        parts / total);
                it.n_parts = last - it.part + 1;
                it.mine = it.part == cta ? 1 : 0;
                it.stop = 0;
                break;
            }
            k = 0; // the cut fell into the item's closing cost
            if (++h == p.Hk) {
                h = 0;
                ++e;
            }
        }
        if (!it.stop) {
            it.kvh = h;
            it.L = en.L;
            it.key_lo = en.key_lo;
            it.pair = en.n_tok > p.TQ;
            it.u_lo = en.lo + k;
            it.u_hi = en.lo + k_end;
            it.step = it.pair ? 1 : 2;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int blk = it.pair ? t : 0; // the slot's row block
                const int n = min(p.TQ, en.n_tok - blk * p.TQ);
                it.t0[t] = en.t0 + blk * p.TQ;
                it.pos0[t] = en.pos0 + blk * p.TQ;
                it.rows[t] = n * p.G;
                int k0, k1;
                key_range(p, en.L, it.pos0[t], it.pos0[t] + n - 1, k0, k1);
                it.first[t] = max(it.u_lo, k0 / kBN) + (it.pair ? 0 : t);
                it.hi[t] = min(it.u_hi, (max(k1, 0) + kBN - 1) / kBN);
            }
        }
        const uint32_t ring = item_count & 1, slot = item_count % kInfo;
        ok = warp_wait(bar(sm.info_empty[slot]), ((item_count / kInfo) & 1) ^ 1, cx.wc, W_INFO_EMPTY);
        if (!ok)
            break;
        if (lane == 0) {
            sm.info[slot] = it;
            ptx::mbar_arrive(bar(sm.info_full[slot])); // release: the fields above first
        }
        __syncwarp();
        if (it.stop)
            break;
        // ---- Q
        if (item_count >= 2) {
            ok = warp_wait(bar(sm.q_empty[ring]), ((item_count - 2) >> 1) & 1, cx.wc, W_Q_EMPTY);
            if (!ok)
                break;
        }
        if (lane == 0) {
            const int slots = it.pair ? 2 : 1;
            ptx::mbar_arrive_expect_tx(bar(sm.q_full[ring]),
                                       static_cast<uint32_t>(slots * C::kHalves * p.TQ * p.G) * C::kRowBytes);
            for (int t = 0; t < slots; ++t)
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                    ptx::tma_load_4d(ptx::smem_u32(sm.q[ring][t]) + hf * C::kQHalf, tm_q, bar(sm.q_full[ring]),
                                     hf * 64, 0, it.kvh, it.t0[t]);
        }
        __syncwarp();
        ++item_count;
        // ---- K/V: lane g loads the tile's g-th box of 16 keys; its page is
        // fetched a tile ahead
        const int64_t row = static_cast<int64_t>(en.b) * p.bt_stride;
        auto page_of = [&](int j) {
            const int key = j * kBN + static_cast<int>(lane) * kBox;
            if (lane >= kBoxes || key >= it.L)
                return 0;
            return p.page_shift < 0 ? en.b : __ldg(p.block_table + row + (key >> p.page_shift));
        };
        int page_next = page_of(it.u_lo);
        for (int j = it.u_lo; j < it.u_hi; ++j, ++kv_count) {
            const int page = page_next;
            if (j + 1 < it.u_hi)
                page_next = page_of(j + 1);
            const uint32_t s = kv_count % kStages;
            ok = warp_wait(bar(sm.kv_empty[s]), ((kv_count / kStages) & 1) ^ 1, cx.wc, W_KV_EMPTY);
            if (!ok)
                break;
            const int left = it.L - j * kBN;
            const int boxes = left <= 0 ? 0 : min(kBoxes, (left + kBox - 1) / kBox);
            const uint32_t b_full = bar(sm.kv_full[s]);
            if (lane == 0)
                ptx::mbar_arrive_expect_tx(b_full,
                                           static_cast<uint32_t>(2 * C::kHalves * boxes * kBox) * C::kRowBytes);
            __syncwarp();
            if (static_cast<int>(lane) < boxes) {
                const int key = j * kBN + static_cast<int>(lane) * kBox;
                const int at = p.page_shift < 0 ? key : key & ((1 << p.page_shift) - 1);
                const uint32_t off = lane * kBox * C::kRowBytes;
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf) {
                    ptx::tma_load_4d(ptx::smem_u32(sm.k[s]) + hf * C::kKVHalf + off, tm_k, b_full, hf * 64, at,
                                     it.kvh, page);
                    ptx::tma_load_4d(ptx::smem_u32(sm.v[s]) + hf * C::kKVHalf + off, tm_v, b_full, hf * 64, at,
                                     it.kvh, page);
                }
            }
            __syncwarp();
        }
        if (!ok)
            break;
        // ---- on to the next item
        k = 0;
        if (++h == p.Hk) {
            h = 0;
            ++e;
        }
    }
    if (!ok) {
        // wait (bounded, ignoring the abort) for this warp's own loads in flight
        const uint32_t first = kv_count > kStages ? kv_count - kStages : 0;
        for (uint32_t idx = first; idx < kv_count; ++idx)
            mbar_wait_drain(bar(sm.kv_full[idx % kStages]), (idx / kStages) & 1, cx.wc, W_DRAIN);
        for (uint32_t n = item_count > 2 ? item_count - 2 : 0; n < item_count; ++n)
            mbar_wait_drain(bar(sm.q_full[n & 1]), (n >> 1) & 1, cx.wc, W_DRAIN);
    }
}

// ------------------------------------------------------------------ MMA issuers

// The slot's tile among [u_lo, u_hi)?
__device__ __forceinline__ bool uses(int j, int first, int hi, int step)
{
    return j >= first && j < hi && ((j - first) & (step - 1)) == 0;
}

template <int D>
__device__ void s_role(const KernelCtx<D> &cx)
{
    using C = ChunkCfg<D>;
    constexpr int kBN = C::kBN, kStages = C::kStages;
    ChunkSmem<D> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    constexpr uint32_t idesc_qk = umma_idesc_bf16(BM, kBN, false);
    constexpr uint64_t kHiK = umma_desc_hi(16, C::kGroupBytes, kSwizzle128B); // Q, K: K-major
    constexpr uint32_t kTileLo = C::kTileBytes >> 4, kKVLo = C::kKVBytes >> 4;
    const uint32_t q_lo0 = ptx::smem_u32(sm.q[0][0]) >> 4;
    const uint32_t k_lo0 = ptx::smem_u32(sm.k[0]) >> 4;
    uint32_t idx = 0, issued[2] = {0u, 0u};
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t ring = n & 1;
        const uint32_t slot = n % kInfo;
        ok = warp_wait(bar(sm.info_full[slot]), (n / kInfo) & 1, cx.wc, W_INFO_FULL);
        if (!ok)
            break;
        const Item &inf = sm.info[slot];
        const int stop = inf.stop, pair = inf.pair, u_lo = inf.u_lo, u_hi = inf.u_hi, step = inf.step;
        const int first0 = inf.first[0], first1 = inf.first[1], hi0 = inf.hi[0], hi1 = inf.hi[1];
        const int L = inf.L, key_lo = inf.key_lo;
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(bar(sm.info_empty[slot]));
        if (stop)
            break;
        ok = warp_wait(bar(sm.q_full[ring]), (n >> 1) & 1, cx.wc, W_Q_FULL);
        if (!ok)
            break;
        for (int j = u_lo; j < u_hi; ++j, ++idx) {
            const uint32_t stage = idx % kStages;
            ok = warp_wait(bar(sm.kv_full[stage]), (idx / kStages) & 1, cx.wc, W_KV_FULL);
            if (!ok)
                break;
            // rows of V that no query row sees: zero (their P is 0, but the bytes
            // may be anything).  Each lane's writes reach the tensor core through
            // its proxy fence, s_full, p_full and the P V issue.
            const int j0 = j * kBN;
            const int dead_lo = min(kBN, max(0, key_lo - j0)), dead_hi = min(kBN, max(0, L - j0));
            if (dead_lo > 0 || dead_hi < kBN) {
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf) {
                    uint4 *v = reinterpret_cast<uint4 *>(sm.v[stage] + hf * C::kKVHalf);
                    for (int c = lane; c < dead_lo * 8; c += 32)
                        v[c] = make_uint4(0, 0, 0, 0);
                    for (int c = dead_hi * 8 + lane; c < kBN * 8; c += 32)
                        v[c] = make_uint4(0, 0, 0, 0);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
            }
            const uint32_t klo = k_lo0 + stage * kKVLo;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!uses(j, t ? first1 : first0, t ? hi1 : hi0, step))
                    continue;
                if (issued[t] > 0) {
                    // the softmax has copied the slot's previous S out of TMEM
                    ok = warp_wait(bar(sm.s_free[t]), (issued[t] - 1) & 1, cx.wc, W_S_FULL);
                    if (!ok)
                        break;
                }
                ++issued[t];
                ptx::tc_fence_after();
                if (lane == 0) {
                    const uint32_t qlo = q_lo0 + (2 * ring + (pair ? t : 0)) * kTileLo;
                    const uint32_t tS = cx.tmem + C::kColS + C::kStrideS * t;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t qo = (kk / 4) * (C::kQHalf >> 4) + 2 * (kk % 4);
                        const uint32_t ko = (kk / 4) * (C::kKVHalf >> 4) + 2 * (kk % 4);
                        ptx::mma_ss(tS, kHiK | (qlo + qo), kHiK | (klo + ko), idesc_qk, kk > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(bar(sm.s_full[t]));
                }
                __syncwarp();
            }
            if (!ok)
                break;
        }
        if (!ok)
            break;
        if (lane == 0)
            ptx::mma_commit(bar(sm.q_empty[ring])); // every read of this Q buffer issued so far
        __syncwarp();
    }
    // every MMA this thread issued has completed before TMEM is released
    const uint32_t b_final = bar(sm.final_bar[0]);
    if (lane == 0)
        ptx::mma_commit(b_final);
    __syncwarp();
    mbar_wait_drain(b_final, 0, cx.wc, W_FINAL);
}

template <int D>
__device__ void pv_role(const KernelCtx<D> &cx, int t)
{
    using C = ChunkCfg<D>;
    constexpr int kBN = C::kBN, kStages = C::kStages;
    ChunkSmem<D> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    constexpr uint32_t idesc_pv = umma_idesc_bf16(BM, C::kDvExt, true);
    constexpr uint32_t kKVLo = C::kKVBytes >> 4;
    const uint32_t v_lo0 = ptx::smem_u32(sm.v[0]) >> 4;
    const uint32_t ones_lo = ptx::smem_u32(sm.ones) >> 4;
    const uint32_t tO = cx.tmem + C::kColO + C::kStrideO * t;
    const uint32_t tP = cx.tmem + C::kColP + C::kStrideP * t;
    uint32_t idx = 0, pcount = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kInfo;
        ok = warp_wait(bar(sm.info_full[slot]), (n / kInfo) & 1, cx.wc, W_INFO_FULL);
        if (!ok)
            break;
        const Item &inf = sm.info[slot];
        const int stop = inf.stop, u_lo = inf.u_lo, u_hi = inf.u_hi, step = inf.step;
        const int first = inf.first[t], hi = inf.hi[t];
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(bar(sm.info_empty[slot]));
        if (stop)
            break;
        for (int j = u_lo; j < u_hi; ++j, ++idx) {
            const uint32_t stage = idx % kStages;
            if (!uses(j, first, hi, step)) {
                // tile not used by this slot: release it once it has landed
                ok = warp_wait(bar(sm.kv_full[stage]), (idx / kStages) & 1, cx.wc, W_KV_FULL);
                if (!ok)
                    break;
                if (lane == 0)
                    ptx::mbar_arrive(bar(sm.kv_empty[stage]));
                __syncwarp();
                continue;
            }
            ok = warp_wait(bar(sm.p_full[t]), pcount & 1, cx.wc, W_P_FULL);
            if (!ok)
                break;
            ++pcount;
            ptx::tc_fence_after();
            if (lane == 0) {
                // D = 64: O += P [V_j | 1] (V's second column block is the ones
                // tile, LBO bytes away); D = 128: V's two 64-column halves
                const uint32_t vlo = v_lo0 + stage * kKVLo;
                const uint32_t lbo = C::kOnes ? (ones_lo - vlo) << 4 : C::kKVHalf;
                const uint64_t hi_v = umma_desc_hi(lbo, C::kGroupBytes, kSwizzle128B);
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)
                    ptx::mma_ts(tO, tP + 8 * kk, hi_v | (vlo + kk * (16 * C::kRowBytes >> 4)), idesc_pv,
                                (j > first || kk > 0) ? 1u : 0u);
                ptx::mma_commit(bar(sm.pv_done[t]));
                ptx::mma_commit(bar(sm.kv_empty[stage]));
            }
            __syncwarp();
        }
    }
    const uint32_t b_final = bar(sm.final_bar[1 + t]);
    if (lane == 0)
        ptx::mma_commit(b_final);
    __syncwarp();
    mbar_wait_drain(b_final, 0, cx.wc, W_FINAL);
}

// ------------------------------------------------------------------ softmax

// 16 columns of a row's output: normalised, bf16, two 16-byte stores.
__device__ __forceinline__ void store16(__nv_bfloat16 *dst, const float (&o)[16], float inv)
{
    uint4 *d = reinterpret_cast<uint4 *>(dst);
#pragma unroll
    for (int c = 0; c < 2; ++c)
        d[c] = make_uint4(ptx::pack_bf16(o[8 * c] * inv, o[8 * c + 1] * inv),
                          ptx::pack_bf16(o[8 * c + 2] * inv, o[8 * c + 3] * inv),
                          ptx::pack_bf16(o[8 * c + 4] * inv, o[8 * c + 5] * inv),
                          ptx::pack_bf16(o[8 * c + 6] * inv, o[8 * c + 7] * inv));
}

// Joins the parts of the item's rows 32 w .. 32 w + 31 (columns [col0, col0 +
// N) of the output; each part holds them as N fp32 columns of 128 rows, then
// m, l and the sum of the rounded P).  Whole warp.  Lanes are spread over rows
// first and columns with what is left, so that a single token's few rows use
// the warp as well as 32 rows do.
template <int N, int D>
__device__ __forceinline__ void join_parts(const ChunkParams &p, int slot, int part, int n_parts, int rows, int w,
                                           int t0, int kvh, int col0, bool with_lse)
{
    const int lane = static_cast<int>(ptx::lane_id());
    const int n = min(32, rows - 32 * w);
    int span = 1;
    while (span < n)
        span *= 2;
    const int r = 32 * w + (lane & (span - 1));
    const int cstep = 32 / span, c_first = lane / span;
    const bool live = r < rows;
    // part q (of CTA part + q) is in that CTA's buffer 1 if the item began there, else 0
    auto base = [&](int q) {
        return p.partials + (static_cast<int64_t>((part + q) * 2 + (q == 0 ? 1 : 0)) * 2 + slot) * ((D + 4) * 128) + r;
    };
    float M = kNegInf, l = 0.f, lr = 0.f;
    if (live)
        for (int q = 0; q < n_parts; ++q)
            M = fmaxf(M, __ldcg(base(q) + N * 128));
    if (live && M != kNegInf)
        for (int q = 0; q < n_parts; ++q) {
            const float *b = base(q) + N * 128;
            const float wq = ptx::ex2(__ldcg(b) - M);
            l = fmaf(wq, __ldcg(b + 128), l);
            lr = fmaf(wq, __ldcg(b + 256), lr);
        }
    const float inv = lr > 0.f ? ptx::rcp_approx(lr) : 0.f;
    const int tok = t0 + fast_div(r, p.div_g), head = kvh * p.G + (r - fast_div(r, p.div_g) * p.G);
    __nv_bfloat16 *out = p.out + static_cast<int64_t>(tok) * p.o_st + static_cast<int64_t>(head) * p.o_sh + col0;
    for (int c0 = c_first; c0 < N; c0 += 16 * cstep) {
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[i] = 0.f;
        if (live && M != kNegInf)
            for (int q = 0; q < n_parts; ++q) {
                const float *b = base(q);
                const float m = __ldcg(b + N * 128);
                if (m == kNegInf)
                    continue; // a part without a key of this row: its O was not written
                const float wq = ptx::ex2(m - M);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c0 + i * cstep < N)
                        o[i] = fmaf(wq, __ldcg(b + (c0 + i * cstep) * 128), o[i]);
            }
        if (!live)
            continue;
        if (cstep == 1) {
            store16(out + c0, o, inv);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c0 + i * cstep < N)
                    out[c0 + i * cstep] = __float2bfloat16(o[i] * inv);
        }
    }
    if (with_lse && live && c_first == 0 && p.lse)
        p.lse[static_cast<int64_t>(head) * p.l_sh + tok] = l > 0.f ? (M + log2f(l)) * kLn2 : kNegInf;
}

// A row's finished sums and, per part, where it goes.
template <int D>
struct RowOut {
    __nv_bfloat16 *out; // the row's first column
    float *lse;         // null: none
    float *mine;        // this CTA's partial of the row
};

template <int D>
__device__ __forceinline__ RowOut<D> row_out(const ChunkParams &p, const Item &inf, int t, int r)
{
    const int r_tok = fast_div(r, p.div_g);
    const int64_t tok = inf.t0[t] + r_tok, head = inf.kvh * p.G + r - r_tok * p.G;
    RowOut<D> w;
    w.out = p.out + tok * p.o_st + head * p.o_sh;
    w.lse = p.lse ? p.lse + head * p.l_sh + tok : nullptr;
    w.mine = p.partials + (static_cast<int64_t>(blockIdx.x * 2 + inf.mine) * 2 + t) * ((D + 4) * 128) + r;
    return w;
}

// After a warp's partials: the last CTA to come joins the item's parts.
template <int N, int D>
__device__ __forceinline__ void arrive_and_join(const ChunkParams &p, const Item &inf, int t, int wq, int col0,
                                                bool with_lse)
{
    __threadfence();
    __syncwarp();
    int old = 0;
    if (ptx::lane_id() == 0)
        old = atomicAdd(p.tickets + (inf.part * 2 + t) * 4 + wq, 1);
    if (__shfl_sync(0xffffffffu, old, 0) != inf.n_parts - 1)
        return;
    __threadfence();
    join_parts<N, D>(p, t, inf.part, inf.n_parts, inf.rows[t], wq, inf.t0[t], inf.kvh, col0, with_lse);
}

// Epilogue of a pair: the slot's own rows, every column.  An active warp.
template <int D>
__device__ __forceinline__ void write_slot(const ChunkParams &p, const Item &inf, int t, int r, uint32_t tO,
                                           const RowState &st, bool any)
{
    const bool live = r < inf.rows[t], whole = inf.n_parts == 1;
    const RowOut<D> w = row_out<D>(p, inf, t, r);
    const float inv = row_inv_norm(st);
    // an accumulator without a tile, or a row without a key, is not read
    const bool keys = any && st.m_ref != kNegInf;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t raw[32];
        if (any) {
            ptx::tmem_ld32(tO + c, raw);
            ptx::tmem_wait_ld();
            ptx::reg_fence<32>(raw);
        }
        if (!live)
            continue;
        if (whole) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[i] = keys ? __uint_as_float(raw[16 * hf + i]) : 0.f;
                store16(w.out + c + 16 * hf, o, inv);
            }
        } else if (keys) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                __stcg(w.mine + (c + i) * 128, __uint_as_float(raw[i]));
        }
    }
    if (whole) {
        if (live && w.lse)
            *w.lse = row_lse(st);
        return;
    }
    if (live) {
        __stcg(w.mine + D * 128, st.m_ref);
        __stcg(w.mine + (D + 1) * 128, st.l);
        __stcg(w.mine + (D + 2) * 128, st.l_round);
    }
}

// Epilogue of one row block, after both slots are done: this warpgroup's half
// of the columns from both accumulators.  An active warp.
template <int D>
__device__ __forceinline__ void write_joined(const ChunkParams &p, const Item &inf, int t, int r, uint32_t tO,
                                             uint32_t tO_other, uint32_t tX_other, const RowState &st)
{
    constexpr int H = D / 2;
    const bool live = r < inf.rows[t], whole = inf.n_parts == 1;
    const RowOut<D> w = row_out<D>(p, inf, t, r);
    uint32_t other[4];
    ptx::tmem_ld4(tX_other, other);
    ptx::tmem_wait_ld();
    ptx::reg_fence<4>(other);
    const float m1 = __uint_as_float(other[0]), m = fmaxf(st.m_ref, m1);
    const float w0 = st.m_ref == kNegInf ? 0.f : ptx::ex2(st.m_ref - m);
    const float w1 = m1 == kNegInf ? 0.f : ptx::ex2(m1 - m);
    const float l = w0 * st.l + w1 * __uint_as_float(other[1]);
    const float lr = w0 * st.l_round + w1 * __uint_as_float(other[2]);
    const float inv = lr > 0.f ? ptx::rcp_approx(lr) : 0.f;
#pragma unroll 1
    for (int c = 0; c < H; c += 16) {
        uint32_t a[16], b[16];
        float o[16];
        ptx::tmem_ld16(tO + t * H + c, a);
        ptx::tmem_ld16(tO_other + t * H + c, b);
        ptx::tmem_wait_ld();
        ptx::reg_fence<16>(a);
        ptx::reg_fence<16>(b);
#pragma unroll
        for (int i = 0; i < 16; ++i) // an accumulator without a key holds anything
            o[i] = (w0 > 0.f ? w0 * __uint_as_float(a[i]) : 0.f) + (w1 > 0.f ? w1 * __uint_as_float(b[i]) : 0.f);
        if (!live)
            continue;
        if (whole) {
            store16(w.out + t * H + c, o, inv);
        } else if (m != kNegInf) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                __stcg(w.mine + (c + i) * 128, o[i]);
        }
    }
    if (!live)
        return;
    if (whole) {
        if (t == 0 && w.lse)
            *w.lse = l > 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
    } else {
        __stcg(w.mine + H * 128, m);
        __stcg(w.mine + (H + 1) * 128, l);
        __stcg(w.mine + (H + 2) * 128, lr);
    }
}

template <int MOD, int D>
__device__ void softmax_role(const KernelCtx<D> &cx, const ChunkParams &p, int t)
{
    using C = ChunkCfg<D>;
    constexpr int kBN = C::kBN;
    // the warpgroups of a pair take turns on the exponentials of plain scores
    // and run freely with softcap, as in the standard kernel
    constexpr bool kTurns = MOD != MOD_SOFTCAP;
    ChunkSmem<D> &sm = *cx.sm;
    const int r = threadIdx.x & 127;            // row of the block = TMEM lane
    const int wq = (threadIdx.x >> 5) & 3;      // warp's quarter of the lanes
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = cx.tmem + lanes + C::kColS + C::kStrideS * t;
    const uint32_t tO = cx.tmem + lanes + C::kColO + C::kStrideO * t;
    const uint32_t tP = cx.tmem + lanes + C::kColP + C::kStrideP * t;
    const uint32_t b_turn_mine = bar(sm.turn[t]), b_turn_other = bar(sm.turn[t ^ 1]);
    uint32_t scount = 0, pvcount = 0, turns = 0, joins = 0;
    ScoreMod smod;
    smod.qk_log2 = p.qk_log2;
    smod.softcap_in = p.softcap_in;
    smod.softcap_out = p.softcap_out;
    smod.alibi_c = smod.scale = smod.b = smod.h = 0.f;
    auto turn_wait = [&]() {
        return (t == 0 && turns == 0) || warp_wait(b_turn_mine, (t == 1 ? turns : turns - 1) & 1, cx.wc, W_TURN);
    };

    for (uint32_t n = 0;; ++n) {
        if (!warp_wait(bar(sm.info_full[n % kInfo]), (n / kInfo) & 1, cx.wc, W_INFO_FULL))
            return;
        const Item &inf = sm.info[n % kInfo];
        if (inf.stop)
            return;
        const int first = inf.first[t], step = inf.step;
        const int n_mine = inf.hi[t] > first ? (inf.hi[t] - first + step - 1) / step : 0;
        const bool active = 32 * wq < inf.rows[t]; // warp-uniform
        const bool take_turns = kTurns && inf.pair;
        RowState st{kNegInf, 0.f, 0.f};
        if (take_turns) // turns of tiles before this slot's
            for (int j = n_mine ? first - inf.u_lo : inf.u_hi - inf.u_lo; j > 0; --j, ++turns) {
                if (!turn_wait())
                    return;
                ptx::mbar_arrive(b_turn_other);
            }
        if (active) {
            const int pos0 = inf.pos0[t], L = inf.L;
            int row_lo, row_hi, full_lo, full_hi, unused;
            {
                const int pos = pos0 + fast_div(r, p.div_g), last = pos0 + fast_div(inf.rows[t] - 1, p.div_g);
                key_range(p, L, pos, pos, row_lo, row_hi);
                key_range(p, L, last, last, full_lo, unused);
                key_range(p, L, pos0, pos0, unused, full_hi);
            }
            for (int kk = 0; kk < n_mine; ++kk) {
                if (!warp_wait(bar(sm.s_full[t]), scount & 1, cx.wc, W_S_FULL))
                    return;
                ++scount;
                ptx::tc_fence_after();
                float x[kBN];
                load_scores<kBN>(tS, x);
                ptx::tc_fence_before();
                ptx::mbar_arrive(bar(sm.s_free[t])); // S[t] may be overwritten
                if (take_turns && !turn_wait())
                    return;
                const int j0 = (first + kk * step) * kBN;
                apply_score_mod<MOD, kBN>(x, smod, 0, j0);
                if (!(j0 >= full_lo && j0 + kBN <= full_hi))
                    apply_row_mask<kBN>(x, j0, row_lo, row_hi);
                uint32_t pk[kBN / 2];
                bool rescale;
                const float alpha =
                    C::kOnes ? softmax_compute_p_exact_sum<kBN>(x, MOD == MOD_NONE ? p.qk_log2 : 1.f, st, kk == 0,
                                                                pk, rescale)
                             : softmax_compute_p<kBN>(x, MOD == MOD_NONE ? p.qk_log2 : 1.f, st, kk == 0, pk,
                                                      rescale);
                if (take_turns) {
                    ptx::mbar_arrive(b_turn_other); // hand the turn over
                    ++turns;
                }
                if (kk > 0) {
                    // the previous tile's P V has consumed P[t] and landed in O[t]
                    if (!warp_wait(bar(sm.pv_done[t]), pvcount & 1, cx.wc, W_O_FULL))
                        return;
                    ++pvcount;
                    ptx::tc_fence_after();
                    if (rescale)
                        rescale_o<C::kDvExt>(tO, alpha);
                }
                store_p<kBN>(tP, pk);
                ptx::tc_fence_before();
                ptx::mbar_arrive(bar(sm.p_full[t]));
            }
        } else {
            // no row of the item: the hand-offs alone
            for (int kk = 0; kk < n_mine; ++kk) {
                if (!warp_wait(bar(sm.s_full[t]), scount & 1, cx.wc, W_S_FULL))
                    return;
                ++scount;
                ptx::mbar_arrive(bar(sm.s_free[t]));
                if (take_turns) {
                    if (!turn_wait())
                        return;
                    ptx::mbar_arrive(b_turn_other);
                    ++turns;
                }
                if (kk > 0) {
                    if (!warp_wait(bar(sm.pv_done[t]), pvcount & 1, cx.wc, W_O_FULL))
                        return;
                    ++pvcount;
                }
                ptx::mbar_arrive(bar(sm.p_full[t]));
            }
        }
        if (take_turns && n_mine) // turns of tiles after this slot's
            for (int j = inf.u_hi - inf.hi[t]; j > 0; --j, ++turns) {
                if (!turn_wait())
                    return;
                ptx::mbar_arrive(b_turn_other);
            }

        // ---- epilogue
        if (n_mine) {
            if (!warp_wait(bar(sm.pv_done[t]), pvcount & 1, cx.wc, W_O_FULL))
                return;
            ++pvcount;
            ptx::tc_fence_after();
            if constexpr (C::kOnes) {
                uint32_t sum[1];
                ptx::tmem_ld1(tO + C::kColSum, sum);
                ptx::tmem_wait_ld();
                ptx::reg_fence<1>(sum);
                st.l_round = __uint_as_float(sum[0]);
            }
        }
        if (inf.pair) {
            if (active) {
                write_slot<D>(p, inf, t, r, tO, st, n_mine > 0);
                if (inf.n_parts > 1)
                    arrive_and_join<D, D>(p, inf, t, wq, 0, true);
            }
        } else {
            const uint32_t tX = cx.tmem + lanes + C::kColX;
            if (active) {
                const uint32_t ml[8] = {__float_as_uint(st.m_ref), __float_as_uint(st.l),
                                        __float_as_uint(st.l_round), 0, 0, 0, 0, 0};
                ptx::tmem_st8(tX + C::kStrideX * t, ml);
                ptx::tmem_wait_st();
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(sm.x_full[t]));
            if (!warp_wait(bar(sm.x_full[t ^ 1]), joins & 1, cx.wc, W_JOIN))
                return;
            ptx::tc_fence_after();
            if (active)
                write_joined<D>(p, inf, t, r, tO, cx.tmem + lanes + C::kColO + C::kStrideO * (t ^ 1),
                                tX + C::kStrideX * (t ^ 1), st);
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(sm.x_free[t ^ 1])); // the other slot's O and sums have been read
            if (active && inf.n_parts > 1)
                arrive_and_join<D / 2, D>(p, inf, t, wq, t * (D / 2), t == 0);
            // the other warpgroup has read this slot's O before the next item's P V
            if (!warp_wait(bar(sm.x_free[t]), joins & 1, cx.wc, W_JOIN))
                return;
            ptx::tc_fence_after();
            ++joins;
        }
        __syncwarp();
        if (ptx::lane_id() == 0)
            ptx::mbar_arrive(bar(sm.info_empty[n % kInfo]));
    }
}

template <int MOD, int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ChunkParams p)
{
    using C = ChunkCfg<D>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = ptx::smem_u32(smem_raw);
    ChunkSmem<D> *sm = reinterpret_cast<ChunkSmem<D> *>(smem_raw + ((1024u - (base & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5;

    for (uint32_t w = threadIdx.x; w < C::kOnesBytes / 4; w += kThreads)
        reinterpret_cast<uint32_t *>(sm->ones)[w] = 0x3F803F80u; // bf16 1.0 pairs
    ptx::fence_proxy_async_smem();
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar(sm->q_full[b]), 1);
            ptx::mbar_init(bar(sm->q_empty[b]), 1);
        }
        for (int b = 0; b < kInfo; ++b) {
            ptx::mbar_init(bar(sm->info_full[b]), 1);
            ptx::mbar_init(bar(sm->info_empty[b]), 11); // S, two P V and eight softmax warps
        }
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar(sm->kv_full[s]), 1);
            ptx::mbar_init(bar(sm->kv_empty[s]), 2); // one arrival per P V warp
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(bar(sm->s_full[t]), 1);
            ptx::mbar_init(bar(sm->p_full[t]), 128);
            ptx::mbar_init(bar(sm->s_free[t]), 128);
            ptx::mbar_init(bar(sm->pv_done[t]), 1);
            ptx::mbar_init(bar(sm->turn[t]), 128);
            ptx::mbar_init(bar(sm->x_full[t]), 128);
            ptx::mbar_init(bar(sm->x_free[t]), 128);
        }
        for (int b = 0; b < 3; ++b)
            ptx::mbar_init(bar(sm->final_bar[b]), 1);
        sm->abort_flag = 0;
        ptx::fence_mbarrier_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 0 && ptx::lane_id() == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&sm->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();

    KernelCtx<D> cx;
    cx.sm = sm;
    cx.tmem = sm->tmem_base;
    cx.wc.abort_flag = &sm->abort_flag;
    cx.wc.timeout_cycles = p.timeout_ns * 21 / 10; // 2.1 cycles per ns at the maximum clock
    cx.wc.err_user = p.err_user;
    cx.wc.err_lib = &g_lib_error_word;

    // each branch ends with its own copy of the teardown barrier, so no code
    // runs under both register limits
    if (warp >= 4) {
        ptx::setmaxnreg_inc<kRegsSoftmax>();
        softmax_role<MOD, D>(cx, p, (warp >> 2) - 1);
        ptx::tc_fence_before();
        ptx::named_barrier_sync(1, kThreads);
    } else {
        ptx::setmaxnreg_dec<kRegsOther>();
        if (warp == 0)
            producer_role(cx, p, &tm_q, &tm_k, &tm_v);
        else if (warp == 1)
            s_role(cx);
        else
            pv_role(cx, warp - 2);
        ptx::tc_fence_before();
        ptx::named_barrier_sync(1, kThreads);
        if (warp == 1) {
            ptx::tc_fence_after();
            ptx::tmem_dealloc(cx.tmem, 512);
        }
    }
}

template <int MOD, int D>
cudaError_t launch_mod(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const ChunkParams &p,
                       cudaStream_t stream)
{
    // the layout plus the worst-case alignment pad within 227 KB per CTA
    static_assert(sizeof(ChunkSmem<D>) + 1024 <= 232448, "shared memory per CTA");
    const size_t smem = sizeof(ChunkSmem<D>) + 1024;
    static bool configured = false; // benign race: both calls are idempotent
    if (!configured) {
        cudaFuncAttributes attr;
        cudaError_t e = cudaFuncGetAttributes(&attr, chunk_kernel<MOD, D>);
        if (e != cudaSuccess)
            return e;
        // the setmaxnreg split assumes exactly kRegsLaunch registers at launch
        if (attr.numRegs != static_cast<int>(kRegsLaunch))
            return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(chunk_kernel<MOD, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem));
        if (e != cudaSuccess)
            return e;
        configured = true;
    }
    chunk_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    chunk_kernel<MOD, D><<<p.n_cta, kThreads, smem, stream>>>(tq, tk, tv, p);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_chunk(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const ChunkParams &p,
                         cudaStream_t stream)
{
    if (p.head_dim == 64)
        return p.score_mod == MOD_SOFTCAP ? launch_mod<MOD_SOFTCAP, 64>(tq, tk, tv, p, stream)
                                          : launch_mod<MOD_NONE, 64>(tq, tk, tv, p, stream);
    return p.score_mod == MOD_SOFTCAP ? launch_mod<MOD_SOFTCAP, 128>(tq, tk, tv, p, stream)
                                      : launch_mod<MOD_NONE, 128>(tq, tk, tv, p, stream);
}

} // namespace fl
