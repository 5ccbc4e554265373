// chunk_few.cuh -- the few-row path of fwd_chunk.cu: a request whose new
// tokens times the heads of a KV group are at most 16 rows (single tokens,
// drafts) against all of its keys.
//
// Bound by HBM: every key and value is read once and meets a handful of rows.
// So the products are turned round: S^T = K Q^T puts a key in each of the 128
// TMEM lanes and a query row in each of 16 columns, and all lanes of the
// softmax exponentiate however few the rows are (rows in lanes leave 124 of
// 128 idle for a token of a group of four heads: 131 us for 64 requests of 512
// to 8192 keys, 32 heads over 8 of 64, where this takes 101).  P^T goes to shared memory as the B
// operand of O^T = V^T P^T, which accumulates a dimension per lane and a row
// per column.  P goes as two bf16 terms, P rounded and what the rounding left
// (columns of their own, added at the end): with the products this small the
// second term costs nothing, and O keeps the accuracy of an fp32 P.
//
// What matters is bytes in flight: K and V have rings of their own (192 KB in
// all; a K stage is free as soon as S is computed), and the two slots (a
// softmax warpgroup each) take the tiles of two neighbouring KV heads in
// turn, whose rows share DRAM pages and 256-byte L2 fetches (one head after
// the other read 1.48 times the bytes).  An odd last head is slot 0's alone.
//
// Weights are 2^z relative to a fixed reference, 2^0: floating point keeps
// their relative precision wherever they lie, so a running maximum is needed
// against overflow and underflow alone.  A row starts without a reference and
// gets 0 from the first tile that holds a key of it with z >= -kFewRange (one
// bit a row, ORed over the slot's warps); only where a logit exceeds its
// reference by kFewRange, or a row's first keys all lie below, do the warps
// agree on the tile's maximum, rescale and do the tile again.  2^+-60 leaves
// fp32 sums of 2^60 such weights in range, and what lies 2^-66 below a row's
// largest weight does not reach its bf16 output or its LSE.
//
// 64 requests of 8192 keys take 174 to 178 us, 0.9 of the rate of a plain copy; what
// shorter ones pay more is the plan (6 us until it is seen), the first loads
// (5 us), the uneven end (5 us) and the joins (5 us).
//
// A cache in 8 bits (F8) goes through the same products as it is, half the bytes a
// key: tcgen05's kind::f8f6f4 multiplies its e4m3 codes.  Q comes as two e4m3 terms, which
// hold a bf16 number exactly (split_q), and a key's scale, one number per TMEM lane, goes
// into its scores; P goes in f16's precision, as three e5m2 terms with V's scale in it
// (few_item_fp8).  K and V come together, in tiles of 16 KB and one ring: at half the bytes a
// key it is the chain of a tile (S, its softmax, P, the product) that limits, so tiles have 256 keys
// at D = 64 (128: 112 us on the 64 requests above) and a row references for all its keys, which
// move rarely.  64 requests of 512 to 8192 keys take 69 us, of 8192 keys 107 (0.74 of the copy's
// rate); the start (14 us until the first S) and the end (8 us) weigh twice as much here.
//
//   warp  0     walks the CTA's items, publishes them, loads Q, K and V by TMA
//   warp  1     issues S^T of both slots
//   warps 2, 3  issue O^T of slot 0, slot 1, after zeroing V rows that no row sees
//               (or warp 2 both, and warp 3 loads V: few_split_loads; in 8 bits
//               warp 3 walks the items)
//   warps 4-11  the slots' softmax warpgroups
#pragma once

#include <cuda_bf16.h>

#include "chunk_plan.cuh"
#include "fp8.cuh"
#include "softmax_tile.cuh"

namespace fl {
namespace {

constexpr float kFewRange = 60.f; // log2 units

template <int D, bool F8 = false>
struct FewCfg {
    static constexpr int kBN = few_tile(D, F8), kSub = kBN / 128; // keys of a tile, of 128 each
    static constexpr int kHalves = F8 ? 1 : D / 64;
    static constexpr int kStages = F8 ? 5 : D == 128 ? 3 : 6; // of K, and of V
    static constexpr int kLag = F8 ? 0 : D == 128 ? 1 : 2;  // tiles that V is loaded behind K
    static_assert(kLag < kStages, "K of the lag's tiles is loaded before V frees anything");
    static constexpr uint32_t kRowBytes = F8 ? D : 128;     // a row, or 64 columns of it
    static constexpr uint32_t kRowSwizzle = kRowBytes == 64 ? kSwizzle64B : kSwizzle128B;
    static constexpr uint32_t kGroupBytes = 8 * kRowBytes;
    static constexpr uint32_t kQPart = kFewRows * kRowBytes; // half the columns of Q, or one of its two terms
    static constexpr int kQParts = F8 ? 2 : kHalves;
    static constexpr uint32_t kQBytes = kQParts * kQPart;
    static constexpr uint32_t kHalf = kBN * kRowBytes;      // half a K or V tile, or all of it
    static constexpr uint32_t kTileBytes = kHalves * kHalf;
    static constexpr uint32_t kPRow = F8 ? 48 : 64;         // bytes of a key's row of P: two terms (8 bits: three) of up to 16 rows
    // Buffers of a slot's P: the next tile's may be written while this one's product runs
    static constexpr int kPBufs = F8 ? 2 : 1;
    static constexpr uint32_t kColS = 0, kColO = 64, kStride = 32; // TMEM columns of slot t: + 32 t
    static constexpr uint32_t kStrideO = F8 ? 64 : 32;      // (of O)
    static constexpr uint32_t kColumns = F8 ? 256 : 128;
    static constexpr uint32_t kSubS = 16;                   // and of S of the tile's second 128 keys
};

// A CTA's part of an item.  Tiles are numbered as they pass through the
// rings: key tile v >> shift, of head kvh + (v & 1) where shift is 1.
struct FewItem {
    int stop;
    int shift;
    int u_lo, u_hi;       // tiles of this part
    int lo, hi;           // key tiles that any row sees
    int heads;            // KV heads: slots in use
    int t0, rows, pos0;   // first token row, rows, first position
    int L, key_lo;        // cached keys; lowest key that any row sees
    int b, kvh;           // request, (first) KV head
    int n_parts;          // CTAs that share the item; 0: the warm-up
    int cta;              // this part among those of both paths
    int mine;             // its buffer: 1 if the item begins here
};

// The slot's tiles: first, first + step, ... < hi.
struct FewTiles {
    int first, hi, step;
};
__device__ __forceinline__ FewTiles few_tiles(const FewItem &it, int t)
{
    FewTiles f;
    f.first = max(it.u_lo, it.lo << it.shift);
    f.step = 1 << it.shift;
    if (it.shift)
        f.first += (f.first ^ t) & 1;
    f.hi = t < it.heads ? min(it.u_hi, it.hi << it.shift) : 0;
    return f;
}

// A cache in 8 bits: maxima of z - m of each softmax warp, and ref - m, each warp's own.
struct FewSums {
    float most[2][4][kFewRows];
    alignas(16) float gap[2][4][kFewRows];
};

template <int D, bool F8>
struct __align__(1024) FewSmem {
    using C = FewCfg<D, F8>;
    uint8_t k[C::kStages][C::kTileBytes];
    uint8_t v[C::kStages][C::kTileBytes];
    uint8_t q[2][2][C::kQBytes];     // [Q buffer][slot]
    uint8_t p[2][C::kPBufs][C::kBN * C::kPRow]; // [slot]
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[C::kStages], k_empty[C::kStages];
    uint64_t v_full[F8 ? 1 : C::kStages], v_empty[F8 ? 1 : C::kStages]; // (in 8 bits V comes with K)
    uint64_t s_full[2], s_free[2], p_full[2][C::kPBufs], pv_done[2][C::kPBufs];
    uint64_t group[2];               // the slot's softmax warps among themselves
    uint64_t final_bar[3];
    uint64_t info_full[kInfo], info_empty[kInfo];
    FewItem info[kInfo];
    float red[2][4][kFewRows];       // maxima or sums of each softmax warp
    uint32_t rows[2][2][4];          // by tile parity, of each softmax warp: see few_softmax
    uint32_t large[2][4];            // 8 bits: of tiles in turn, whether a row may ask for a reference
    std::conditional_t<F8, ScaleRing, char> scales;
    std::conditional_t<F8, FewSums, char> sums;
    uint32_t tmem_base;
    uint32_t abort_flag;
};

template <int D, bool F8>
struct FewCtx {
    FewSmem<D, F8> *sm;
    uint32_t tmem;
    int part; // this CTA's place among the parts of the few rows
    WaitCtl wc;
};

// ------------------------------------------------------------------ producers

// A ring of K or V tiles and the one warp that fills it.
template <int D>
struct FewRing {
    using C = FewCfg<D, false>;
    const CUtensorMap *map;
    uint8_t (*tile)[C::kTileBytes];
    uint64_t *full, *empty;
    uint32_t count;

    // Tile v of an item into the next stage: lane g loads the g-th box, of its page.
    __device__ __forceinline__ bool load(const FewCtx<D, false> &cx, const ChunkParams &p, const FewItem &it, int v, int page)
    {
        const int lane = static_cast<int>(ptx::lane_id());
        const int box = 1 << p.few_shift, key0 = (v >> it.shift) * C::kBN, left = it.L - key0;
        const uint32_t s = count % C::kStages;
        if (!warp_wait(bar(empty[s]), ((count / C::kStages) & 1) ^ 1, cx.wc, W_KV_EMPTY))
            return false;
        const int boxes = left <= 0 ? 0 : min(C::kBN >> p.few_shift, (left + box - 1) >> p.few_shift);
        if (lane == 0)
            ptx::mbar_arrive_expect_tx(bar(full[s]), static_cast<uint32_t>(C::kHalves * boxes * box) * C::kRowBytes);
        __syncwarp();
        if (lane < boxes) {
            const int key = key0 + lane * box;
            const int at = p.page_shift < 0 ? key : key & ((1 << p.page_shift) - 1);
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf)
                ptx::tma_load_4d(ptx::smem_u32(tile[s]) + hf * C::kHalf + lane * box * C::kRowBytes, map,
                                 bar(full[s]), hf * 64, at, it.kvh + (it.shift ? v & 1 : 0), page);
        }
        __syncwarp();
        ++count;
        return true;
    }

    // Waits (bounded, ignoring the abort) for the warp's loads in flight.
    __device__ __forceinline__ void drain(const FewCtx<D, false> &cx) const
    {
        for (uint32_t idx = count > C::kStages ? count - C::kStages : 0; idx < count; ++idx)
            mbar_wait_drain(bar(full[idx % C::kStages]), (idx / C::kStages) & 1, cx.wc, W_DRAIN);
    }
};

// Tile v of an item of a cache in 8 bits, the CTA's number `count`: K and V together, with
// their scales.  Lane g loads the g-th box of K, lane 16 + g that of V.
template <int D>
__device__ __forceinline__ bool few_load_fp8(const FewCtx<D, true> &cx, const ChunkParams &p, const CUtensorMap *tm_k,
                                             const CUtensorMap *tm_v, const FewItem &it, int v, uint32_t count, int page)
{
    using C = FewCfg<D, true>;
    FewSmem<D, true> &sm = *cx.sm;
    const int lane = static_cast<int>(ptx::lane_id()), g = lane & 15;
    const int box = 1 << p.few_shift, key0 = (v >> it.shift) * C::kBN, left = it.L - key0;
    const int kvh = it.kvh + (it.shift ? v & 1 : 0);
    const uint32_t s = count % C::kStages, full = bar(sm.k_full[s]);
    if (!warp_wait(bar(sm.k_empty[s]), ((count / C::kStages) & 1) ^ 1, cx.wc, W_KV_EMPTY))
        return false;
    copy_scales<C::kBN / 16>(p, sm.scales, count, full, page, p.few_shift, key0, it.key_lo, it.L, kvh);
    const int boxes = left <= 0 ? 0 : min(C::kBN >> p.few_shift, (left + box - 1) >> p.few_shift);
    if (lane == 0)
        ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(2 * boxes * box) * C::kRowBytes);
    __syncwarp();
    if (g < boxes) {
        const int key = key0 + g * box;
        const int at = p.page_shift < 0 ? key : key & ((1 << p.page_shift) - 1);
        ptx::tma_load_4d(ptx::smem_u32(lane < 16 ? sm.k[s] : sm.v[s]) + g * box * C::kRowBytes, lane < 16 ? tm_k : tm_v,
                         full, 0, at, kvh, page);
    }
    __syncwarp();
    return true;
}

// The page of this lane's box of key tile j.
template <int D, bool F8>
__device__ __forceinline__ int few_page(const ChunkParams &p, const FewItem &it, int j)
{
    const int lane = static_cast<int>(ptx::lane_id()) & (F8 ? 15 : 31), key = j * FewCfg<D, F8>::kBN + (lane << p.few_shift);
    if (lane >= FewCfg<D, F8>::kBN >> p.few_shift || key >= it.L)
        return 0; // never loaded
    return p.page_shift < 0 ? it.b : __ldg(p.block_table + static_cast<int64_t>(it.b) * p.bt_stride + (key >> p.page_shift));
}

// Who loads V: with boxes of 32 keys or more the warp that loads K; with
// smaller ones their number is too much for one warp (pages of 16 keys: 225
// against 178 us for 64 requests of 8192 keys, 128 against 107 of 512 to 8192),
// and V gets the warp that otherwise issues O^T of slot 1, which costs 2 to 7%
// with larger pages (of 32 keys: 108 against 104 us of 512 to 8192).
// (In 8 bits a lane loads a box of each, at once.)
template <bool F8>
__device__ __forceinline__ bool few_split_loads(const ChunkParams &p) { return !F8 && p.few_shift < 5; }

// The next item of the CTA's part from tile k of item h of entry e on (it.stop: none); en, its entry.
template <int D, bool F8>
__device__ __forceinline__ void few_next(const ChunkParams &p, const ChunkPart &me, int cta, int &e, int &h, int &k,
                                         FewItem &it, ChunkEntry &en)
{
    constexpr int kBN = FewCfg<D, F8>::kBN;
    const ChunkEntry *entries = p.entries + p.max_entries;
    int k_end = 0;
    while (e < me.n_entries) {
        en = e == me.entry ? me.at : load_plan(entries + e);
        const int full = item_heads(p, en), heads = min(full, p.Hk - h * full), n_tiles = en.n_tiles * heads;
        const int64_t x0 = en.cum + h * item_cost(p, en);
        if (x0 + static_cast<int64_t>(k) * en.tile_cost >= me.end) {
            e = me.n_entries; // the cut falls before this tile
            break;
        }
        if (k < n_tiles) {
            const PartRange r = part_range<F8>(x0, n_tiles, en.tile_cost, k, me.end, me.total, cta, me.parts);
            k_end = r.k_end;
            it.n_parts = r.n_parts;
            it.mine = r.first == cta ? 1 : 0;
            it.heads = heads;
            it.kvh = h * full;
            it.stop = 0;
            break;
        }
        k = 0; // the cut fell into the item's closing cost
        if (++h * full >= p.Hk) {
            h = 0;
            ++e;
        }
    }
    if (!it.stop) {
        it.shift = it.heads - 1;
        it.cta = me.cta;
        it.u_lo = (en.lo << it.shift) + k;
        it.u_hi = (en.lo << it.shift) + k_end;
        it.b = en.b;
        it.t0 = en.t0;
        it.rows = en.n_tok * p.G;
        it.pos0 = en.pos0;
        it.L = en.L;
        it.key_lo = en.key_lo;
        int k0, k1;
        key_range(p, en.L, en.pos0, en.pos0 + en.n_tok - 1, k0, k1);
        it.lo = k0 / kBN;
        it.hi = (max(k1, 0) + kBN - 1) / kBN;
    }
}

// Walks the CTA's items, publishes them, loads Q, K and, mostly, V.
template <int D>
__device__ void few_producer(const FewCtx<D, false> &cx, const ChunkParams &p, const CUtensorMap *tm_q,
                             const CUtensorMap *tm_k, const CUtensorMap *tm_v)
{
    using C = FewCfg<D, false>;
    FewSmem<D, false> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    FewRing<D> keys{tm_k, sm.k, sm.k_full, sm.k_empty, 0u}, values{tm_v, sm.v, sm.v_full, sm.v_empty, 0u};
    const bool split = few_split_loads<false>(p);
    uint32_t item_count = 0;
    bool ok = true;
    ChunkPart me{};
    const int cta = cx.part;
    int e = 0, h = 0, k = 0; // entry, item of it, tile of that
    bool warm = p.warm;
    if (!warm)
        read_part(p, 1, cta, me, e, h, k);
    for (;;) {
        // ---- the next part
        FewItem it{};
        it.stop = 1;
        ChunkEntry en{};
        // the warm-up, beside the planning kernel: a tile of no keys for each slot, of
        // which nothing is written, so that the roles' instructions are there before
        // the loads begin (behind those of a full GPU they took 12 us)
        if (warm) {
            it.stop = 0;
            it.heads = min(p.Hk, 2);
            it.shift = it.heads - 1;
            it.hi = 1;
            it.u_hi = it.heads;
            it.rows = min(p.G, kFewRows);
        }
        if (!warm)
            few_next<D, false>(p, me, cta, e, h, k, it, en);
        const uint32_t ring = item_count & 1, slot = item_count % kInfo;
        ok = warp_wait(bar(sm.info_empty[slot]), ((item_count / kInfo) & 1) ^ 1, cx.wc, W_INFO_EMPTY);
        if (!ok)
            break;
        if (lane == 0) {
            sm.info[slot] = it;
            ptx::mbar_arrive(bar(sm.info_full[slot])); // release: the fields above first
            if (!it.stop && it.mine && it.n_parts > 1)
                p.joins[me.cta] = ChunkJoin{it.n_parts, JOIN_FEW, it.kvh, {it.t0, it.t0},
                                                {it.rows, it.heads == 2 ? it.rows : 0}, 0};
        }
        __syncwarp();
        if (it.stop)
            break;
        // ---- Q: the rows of each head
        ok = warp_wait(bar(sm.q_empty[ring]), ((item_count >> 1) & 1) ^ 1, cx.wc, W_Q_EMPTY);
        if (!ok)
            break;
        if (lane == 0) {
            const int slots = warm ? 0 : it.heads;
            ptx::mbar_arrive_expect_tx(bar(sm.q_full[ring]),
                                       static_cast<uint32_t>(slots * C::kHalves * p.few_tq * p.G) * C::kRowBytes);
            for (int t = 0; t < slots; ++t)
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                    ptx::tma_load_4d(ptx::smem_u32(sm.q[ring][t]) + hf * C::kQPart, tm_q, bar(sm.q_full[ring]),
                                     hf * 64, 0, it.kvh + t, it.t0);
        }
        __syncwarp();
        ++item_count;
        // ---- K and V: V trails by kLag tiles, as P V trails S, so that it does
        // not wait in shared memory for its weights (not past the item: the next
        // item's buffers may wait for the V of its last tile).  Pages are fetched
        // a tile ahead.
        int page_next = few_page<D, false>(p, it, it.u_lo >> it.shift);
        int page[C::kLag + 1]; // of the last kLag + 1 tiles, the latest first
        for (int v = it.u_lo; v < it.u_hi + (split ? 0 : C::kLag) && ok; ++v) {
#pragma unroll
            for (int i = C::kLag; i > 0; --i)
                page[i] = page[i - 1];
            page[0] = page_next;
            if (v + 1 < it.u_hi)
                page_next = few_page<D, false>(p, it, (v + 1) >> it.shift);
            if (v < it.u_hi)
                ok = keys.load(cx, p, it, v, page[0]);
            if (ok && !split && v - C::kLag >= it.u_lo)
                ok = values.load(cx, p, it, v - C::kLag, page[C::kLag]);
        }
        if (!ok)
            break;
        if (warm) {
            warm = false;
            read_part(p, 1, cta, me, e, h, k);
            continue;
        }
        // ---- on to the next item
        k = 0;
        if (++h * item_heads(p, en) >= p.Hk) {
            h = 0;
            ++e;
        }
    }
    if (!ok) {
        keys.drain(cx);
        values.drain(cx);
        for (uint32_t n = item_count > 2 ? item_count - 2 : 0; n < item_count; ++n)
            mbar_wait_drain(bar(sm.q_full[n & 1]), (n >> 1) & 1, cx.wc, W_DRAIN);
    }
}

// A cache in 8 bits: warp 3 walks the items and publishes them, as far ahead as there is
// room (an item takes it a few microseconds of divisions and loads, which short items'
// loads do not hide), and warp 0 loads them.
template <int D>
__device__ void few_walker_fp8(const FewCtx<D, true> &cx, const ChunkParams &p)
{
    FewSmem<D, true> &sm = *cx.sm;
    ChunkPart me{};
    int e = 0, h = 0, k = 0; // entry, item of it, tile of that
    bool warm = p.warm; // see few_producer
    if (!warm)
        read_part(p, 1, cx.part, me, e, h, k);
    for (uint32_t n = 0;; ++n) {
        FewItem it{};
        ChunkEntry en{};
        if (warm) {
            it.heads = min(p.Hk, 2);
            it.shift = it.heads - 1;
            it.hi = 1;
            it.u_hi = it.heads;
            it.rows = min(p.G, kFewRows);
        } else {
            it.stop = 1;
            few_next<D, true>(p, me, cx.part, e, h, k, it, en);
        }
        const uint32_t slot = n % kInfo;
        if (p.page_shift >= 0 && !it.stop) { // the loader's first look at the block table
            const int key = ((it.u_lo >> it.shift) * FewCfg<D, true>::kBN >> p.page_shift) + static_cast<int>(ptx::lane_id());
            if (key < p.bt_stride)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(p.block_table + static_cast<int64_t>(it.b) * p.bt_stride + key));
        }
        if (!warp_wait(bar(sm.info_empty[slot]), ((n / kInfo) & 1) ^ 1, cx.wc, W_INFO_EMPTY))
            return;
        if (ptx::lane_id() == 0) {
            sm.info[slot] = it;
            ptx::mbar_arrive(bar(sm.info_full[slot])); // release: the fields above first
            if (!it.stop && it.mine && it.n_parts > 1)
                p.joins[me.cta] = ChunkJoin{it.n_parts, JOIN_FEW, it.kvh, {it.t0, it.t0},
                                                {it.rows, it.heads == 2 ? it.rows : 0}, 0};
        }
        __syncwarp();
        if (it.stop)
            return;
        if (warm) {
            warm = false;
            read_part(p, 1, cx.part, me, e, h, k);
            continue;
        }
        k = 0;
        if (++h * item_heads(p, en) >= p.Hk) {
            h = 0;
            ++e;
        }
    }
}

template <int D>
__device__ void few_loader_fp8(const FewCtx<D, true> &cx, const ChunkParams &p, const CUtensorMap *tm_q,
                               const CUtensorMap *tm_k, const CUtensorMap *tm_v)
{
    using C = FewCfg<D, true>;
    FewSmem<D, true> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    uint32_t kv_count = 0, n = 0;
    bool ok = true, fenced = false;
    for (;; ++n) {
        const uint32_t slot = n % kInfo, ring = n & 1;
        ok = warp_wait(bar(sm.info_full[slot]), (n / kInfo) & 1, cx.wc, W_INFO_FULL);
        if (!ok)
            break;
        const FewItem it = sm.info[slot];
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(bar(sm.info_empty[slot]));
        if (it.stop)
            break;
        int page_next = few_page<D, true>(p, it, it.u_lo >> it.shift);
        ok = warp_wait(bar(sm.q_empty[ring]), ((n >> 1) & 1) ^ 1, cx.wc, W_Q_EMPTY);
        if (!ok)
            break;
        if (lane == 0) {
            const int slots = it.n_parts ? it.heads : 0; // none for the warm-up
            if (slots && !fenced)
                ptx::fence_proxy_async_all(); // Q's terms, which the planning kernel has written
            fenced = slots;
            ptx::mbar_arrive_expect_tx(bar(sm.q_full[ring]),
                                       static_cast<uint32_t>(slots * C::kQParts * p.few_tq * p.G) * C::kRowBytes);
            for (int t = 0; t < slots; ++t)
#pragma unroll
                for (int i = 0; i < C::kQParts; ++i)
                    ptx::tma_load_4d(ptx::smem_u32(sm.q[ring][t]) + i * C::kQPart, tm_q, bar(sm.q_full[ring]), 0, 0,
                                     it.kvh + t, it.t0 + i * p.T);
        }
        __syncwarp();
        for (int v = it.u_lo; v < it.u_hi; ++v, ++kv_count) {
            const int page = page_next;
            if (v + 1 < it.u_hi)
                page_next = few_page<D, true>(p, it, (v + 1) >> it.shift);
            ok = few_load_fp8(cx, p, tm_k, tm_v, it, v, kv_count, page);
            if (!ok)
                break;
        }
        if (!ok) {
            ++n;
            break;
        }
    }
    if (!ok) { // wait (bounded, ignoring the abort) for the loads in flight
        for (uint32_t idx = kv_count > C::kStages ? kv_count - C::kStages : 0; idx < kv_count; ++idx)
            mbar_wait_drain(bar(sm.k_full[idx % C::kStages]), (idx / C::kStages) & 1, cx.wc, W_DRAIN);
        for (uint32_t i = n > 2 ? n - 2 : 0; i < n; ++i)
            mbar_wait_drain(bar(sm.q_full[i & 1]), (i >> 1) & 1, cx.wc, W_DRAIN);
    }
}

// Loads V alone (few_split_loads).
template <int D>
__device__ void few_v_producer(const FewCtx<D, false> &cx, const ChunkParams &p, const CUtensorMap *tm_v)
{
    FewSmem<D, false> &sm = *cx.sm;
    FewRing<D> values{tm_v, sm.v, sm.v_full, sm.v_empty, 0u};
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kInfo;
        ok = warp_wait(bar(sm.info_full[slot]), (n / kInfo) & 1, cx.wc, W_INFO_FULL);
        if (!ok)
            break;
        const FewItem it = sm.info[slot];
        __syncwarp();
        if (ptx::lane_id() == 0)
            ptx::mbar_arrive(bar(sm.info_empty[slot]));
        if (it.stop)
            return;
        int page_next = few_page<D, false>(p, it, it.u_lo >> it.shift);
        for (int v = it.u_lo; v < it.u_hi && ok; ++v) {
            const int page = page_next;
            if (v + 1 < it.u_hi)
                page_next = few_page<D, false>(p, it, (v + 1) >> it.shift);
            ok = values.load(cx, p, it, v, page);
        }
    }
    values.drain(cx);
}

// ------------------------------------------------------------------ MMA issuers

template <int D, bool F8>
__device__ void few_s_role(const FewCtx<D, F8> &cx)
{
    using C = FewCfg<D, F8>;
    constexpr int kBN = C::kBN, kStages = C::kStages;
    FewSmem<D, F8> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    constexpr uint32_t idesc = F8 ? umma_idesc_e4m3(128, kFewRows) : umma_idesc_bf16(kBN, kFewRows, false);
    constexpr uint64_t kHi = umma_desc_hi(16, C::kGroupBytes, C::kRowSwizzle); // Q, K: K-major
    const uint32_t q_lo0 = ptx::smem_u32(sm.q[0][0]) >> 4, k_lo0 = ptx::smem_u32(sm.k[0]) >> 4;
    uint32_t idx = 0, issued[2] = {0u, 0u};
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t ring = n & 1, slot = n % kInfo;
        ok = warp_wait(bar(sm.info_full[slot]), (n / kInfo) & 1, cx.wc, W_INFO_FULL);
        if (!ok)
            break;
        const FewItem &inf = sm.info[slot];
        const int stop = inf.stop, shift = inf.shift, u_lo = inf.u_lo, u_hi = inf.u_hi;
        const int lo = inf.lo << shift, hi = inf.hi << shift;
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(bar(sm.info_empty[slot]));
        if (stop)
            break;
        ok = warp_wait(bar(sm.q_full[ring]), (n >> 1) & 1, cx.wc, W_Q_FULL);
        if (!ok)
            break;
        for (int v = u_lo; v < u_hi; ++v, ++idx) {
            const uint32_t stage = idx % kStages, phase = (idx / kStages) & 1;
            const int t = shift ? v & 1 : 0;
            ok = warp_wait(bar(sm.k_full[stage]), phase, cx.wc, W_KV_FULL);
            if (!ok)
                break;
            if (v < lo || v >= hi) { // a tile that no row sees
                if (lane == 0)
                    ptx::mbar_arrive(bar(sm.k_empty[stage]));
                __syncwarp();
                continue;
            }
            if (issued[t] > 0) {
                // the softmax has copied the slot's previous S out of TMEM
                ok = warp_wait(bar(sm.s_free[t]), (issued[t] - 1) & 1, cx.wc, W_S_FULL);
                if (!ok)
                    break;
            }
            ++issued[t];
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t qlo = q_lo0 + (2 * ring + t) * (C::kQBytes >> 4);
                const uint32_t klo = k_lo0 + stage * (C::kTileBytes >> 4);
                const uint32_t tS = cx.tmem + C::kColS + C::kStride * t;
                if constexpr (F8) { // both terms of Q with the same K
#pragma unroll
                    for (int sub = 0; sub < C::kSub; ++sub)
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            ptx::mma_ss_f8(tS + sub * C::kSubS,
                                           kHi | (klo + sub * (128 * C::kRowBytes >> 4) + 2 * (kk % (D / 32))),
                                           kHi | (qlo + kk / (D / 32) * (C::kQPart >> 4) + 2 * (kk % (D / 32))), idesc,
                                           kk > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        ptx::mma_ss(tS, kHi | (klo + (kk / 4) * (C::kHalf >> 4) + 2 * (kk % 4)),
                                    kHi | (qlo + (kk / 4) * (C::kQPart >> 4) + 2 * (kk % 4)), idesc, kk > 0 ? 1u : 0u);
                }
                ptx::mma_commit(bar(sm.s_full[t]));
                ptx::mma_commit(bar(sm.k_empty[stage]));
            }
            __syncwarp();
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

// Issues O^T of the slots from `slot` on: both, or one.  Every warp of this role
// passes every tile in order (and releases what is not its own), so that none
// is ever a turn of the ring away from a barrier whose parity it waits for.
template <int D, bool F8>
__device__ void few_pv_role(const FewCtx<D, F8> &cx, int slot_lo, int slot_hi)
{
    using C = FewCfg<D, F8>;
    constexpr int kBN = C::kBN, kStages = C::kStages;
    FewSmem<D, F8> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    uint64_t *const full = F8 ? sm.k_full : sm.v_full, *const empty = F8 ? sm.k_empty : sm.v_empty;
    // O^T = V^T P^T: both operands with their long index contiguous.  V^T has
    // 128 rows: at D = 64 the second 64 repeat the first (block stride 0).  P
    // has 64-byte rows of a key, 64-byte swizzle.
    // In 8 bits V^T's rows are 64 or 128 bytes, swizzled over their length, and P (e5m2) is
    // not: units of 16 bytes, those of a key kBN * 16 bytes apart.
    constexpr uint32_t kMajor = 1u << 15 | 1u << 16;
    constexpr uint32_t idesc4 = umma_idesc_e4m3_e5m2(128, 16) | kMajor; // F8 alone
    constexpr uint32_t idesc8 = (F8 ? umma_idesc_e4m3_e5m2(128, 32) : umma_idesc_bf16(128, 16, true)) | kMajor;
    constexpr uint32_t idesc16 = (F8 ? umma_idesc_e4m3_e5m2(128, 48) : umma_idesc_bf16(128, 32, true)) | kMajor;
    constexpr uint64_t kHiV = umma_desc_hi(D == 128 ? C::kHalf : 0, C::kGroupBytes, C::kRowSwizzle);
    constexpr uint64_t kHiP = F8 ? umma_desc_hi(8 * 16, kBN * 16, kSwizzleNone) : umma_desc_hi(16, 8 * C::kPRow, kSwizzle64B);
    constexpr int kKeys = F8 ? 32 : 16; // of an MMA
    constexpr uint32_t kPKey = F8 ? 16 : C::kPRow; // bytes from one key to the next
    const uint32_t v_lo0 = ptx::smem_u32(sm.v[0]) >> 4, p_lo0 = ptx::smem_u32(sm.p[0][0]) >> 4;
    uint32_t idx = 0, pcount[2] = {0u, 0u};
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kInfo;
        ok = warp_wait(bar(sm.info_full[slot]), (n / kInfo) & 1, cx.wc, W_INFO_FULL);
        if (!ok)
            break;
        const FewItem &inf = sm.info[slot];
        const int stop = inf.stop, shift = inf.shift, u_lo = inf.u_lo, u_hi = inf.u_hi;
        const int lo = inf.lo << shift, hi = inf.hi << shift, L = inf.L, key_lo = inf.key_lo;
        const int first = max(u_lo, lo);
        const uint32_t idesc = F8 && inf.rows <= 4 ? idesc4 : inf.rows <= 8 ? idesc8 : idesc16; // two or three terms a row
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(bar(sm.info_empty[slot]));
        if (stop)
            break;
        for (int v = u_lo; v < u_hi; ++v, ++idx) {
            const uint32_t stage = idx % kStages;
            const int t = shift ? v & 1 : 0, j0 = (v >> shift) * kBN;
            ok = warp_wait(bar(full[stage]), (idx / kStages) & 1, cx.wc, W_KV_FULL);
            if (!ok)
                break;
            if (v < lo || v >= hi || t < slot_lo || t > slot_hi) {
                // no row sees it, or another warp's
                if (lane == 0)
                    ptx::mbar_arrive(bar(empty[stage]));
                __syncwarp();
                continue;
            }
            // rows of V that no query row sees: zero (their P is 0, but the bytes
            // may be anything)
            const int dead_lo = min(kBN, max(0, key_lo - j0)), dead_hi = min(kBN, max(0, L - j0));
            if (dead_lo > 0 || dead_hi < kBN) {
                constexpr int kUnits = C::kRowBytes / 16;
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf) {
                    uint4 *dst = reinterpret_cast<uint4 *>(sm.v[stage] + hf * C::kHalf);
                    for (int c = lane; c < dead_lo * kUnits; c += 32)
                        dst[c] = make_uint4(0, 0, 0, 0);
                    for (int c = dead_hi * kUnits + lane; c < kBN * kUnits; c += 32)
                        dst[c] = make_uint4(0, 0, 0, 0);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
            }
            const uint32_t buf = pcount[t] % C::kPBufs; // of P
            ok = warp_wait(bar(sm.p_full[t][buf]), (pcount[t] / C::kPBufs) & 1, cx.wc, W_P_FULL);
            if (!ok)
                break;
            ++pcount[t];
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t vlo = v_lo0 + stage * (C::kTileBytes >> 4), plo = p_lo0 + (t * C::kPBufs + buf) * (kBN * C::kPRow >> 4);
                const bool begun = v - first >= 1 << shift; // not the slot's first tile
#pragma unroll
                for (int kk = 0; kk < kBN / kKeys; ++kk)
                    (F8 ? ptx::mma_ss_f8 : ptx::mma_ss)(
                        cx.tmem + C::kColO + C::kStrideO * t, kHiV | (vlo + kk * (kKeys * C::kRowBytes >> 4)),
                        kHiP | (plo + kk * (kKeys * kPKey >> 4)), idesc, (begun || kk > 0) ? 1u : 0u);
                ptx::mma_commit(bar(sm.pv_done[t][buf]));
                ptx::mma_commit(bar(empty[stage]));
            }
            __syncwarp();
        }
    }
    const uint32_t b_final = bar(sm.final_bar[1 + slot_lo]);
    if (lane == 0)
        ptx::mma_commit(b_final);
    __syncwarp();
    mbar_wait_drain(b_final, 0, cx.wc, W_FINAL);
}

// ------------------------------------------------------------------ softmax

// A float's order as a signed integer's.
__device__ __forceinline__ int ordered(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// This thread's weights, 2^(c x - m) (an unset reference counts as 0).
template <int R>
__device__ __forceinline__ void few_exp(const float (&x)[R], float c, const float (&m)[R], bool zero, float (&w)[R])
{
    if (zero) { // every reference is 0
#pragma unroll
        for (int n = 0; n < R; ++n)
            w[n] = ptx::ex2(x[n] * c);
    } else {
#pragma unroll
        for (int n = 0; n < R; ++n)
            w[n] = ptx::ex2(fmaf(x[n], c, m[n] == kNegInf ? 0.f : -m[n]));
    }
}

// O^T's columns of a slot: the rows' sums of rounded weights, then those of the rests.
template <int R>
__device__ __forceinline__ void few_load_o(uint32_t tO, uint32_t (&o)[2 * R])
{
    if constexpr (R == 8)
        ptx::tmem_ld16(tO, o);
    else
        ptx::tmem_ld32(tO, o);
    ptx::tmem_wait_ld();
    ptx::reg_fence<2 * R>(o);
}

// What a softmax thread carries from item to item.
struct FewState {
    uint32_t s, pv, group, tiles; // phases of s_full, pv_done, group; tiles so far
};

// One item of at most R rows.  False when a wait ran out.
template <int MOD, int D, int R>
__device__ __forceinline__ bool few_item(const FewCtx<D, false> &cx, const ChunkParams &p, const FewItem &inf, int t,
                                         FewState &ct)
{
    using C = FewCfg<D, false>;
    constexpr int kBN = C::kBN;
    FewSmem<D, false> &sm = *cx.sm;
    const int r = threadIdx.x & 127; // key of the tile = TMEM lane of S^T; of O^T: dimension
    const int wq = (threadIdx.x >> 5) & 3, lane = static_cast<int>(ptx::lane_id());
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = cx.tmem + lanes + C::kColS + C::kStride * t;
    const uint32_t tO = cx.tmem + lanes + C::kColO + C::kStrideO * t;
    const uint32_t b_group = bar(sm.group[t]);
    const float c = MOD == MOD_NONE ? p.qk_log2 : 1.f;
    ScoreMod smod;
    smod.qk_log2 = p.qk_log2;
    smod.softcap_in = p.softcap_in;
    smod.softcap_out = p.softcap_out;
    smod.alibi_c = smod.scale = smod.b = smod.h = 0.f;
    // 64-byte swizzle: 16-byte unit u of key r at u ^ (r / 2 mod 4)
    uint4 *const pdst = reinterpret_cast<uint4 *>(sm.p[t][0] + r * C::kPRow);
    const int sw = (r >> 1) & 3;
    auto group_sync = [&]() {
        ptx::mbar_arrive(b_group);
        return warp_wait(b_group, ct.group++ & 1, cx.wc, W_JOIN);
    };
    const FewTiles f = few_tiles(inf, t);
    const int n_mine = f.hi > f.first ? (f.hi - f.first + f.step - 1) / f.step : 0;
    const int rows = inf.rows, pos0 = inf.pos0;
    const uint32_t row_bits = (1u << rows) - 1;
    int full_lo, full_hi, unused;
    {
        const int last = pos0 + fast_div(rows - 1, p.div_g);
        key_range(p, inf.L, last, last, full_lo, unused);
        key_range(p, inf.L, pos0, pos0, unused, full_hi);
    }
    float m[R], l[R];
#pragma unroll
    for (int n = 0; n < R; ++n) {
        m[n] = kNegInf;
        l[n] = 0.f;
    }
    uint32_t set = 0;  // rows that have a reference
    bool moved = false; // some reference is not 0
    for (int kk = 0; kk < n_mine; ++kk) {
        if (!warp_wait(bar(sm.s_full[t]), ct.s & 1, cx.wc, W_S_FULL))
            return false;
        ++ct.s;
        ++ct.tiles;
        ptx::tc_fence_after();
        float x[R];
        {
            uint32_t raw[R];
            if constexpr (R == 8)
                ptx::tmem_ld8(tS, raw);
            else
                ptx::tmem_ld16(tS, raw);
            ptx::tmem_wait_ld();
            ptx::reg_fence<R>(raw);
#pragma unroll
            for (int n = 0; n < R; ++n)
                x[n] = __uint_as_float(raw[n]);
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(sm.s_free[t]));
        const int j0 = ((f.first + kk * f.step) >> inf.shift) * kBN;
        apply_score_mod<MOD, R>(x, smod, 0, j0);
        if (!(j0 >= full_lo && j0 + kBN <= full_hi)) {
#pragma unroll
            for (int n = 0; n < R; ++n) {
                int lo, hi;
                const int pos = pos0 + fast_div(n, p.div_g);
                key_range(p, inf.L, pos, pos, lo, hi);
                if (j0 + r < lo || j0 + r >= hi)
                    x[n] = kNegInf;
            }
        }
        // bit n: row n has a key here with z >= -kFewRange; bit 16 + n: one too large
        // for the row's reference, or too small to be its first.  Once every row
        // has the reference 0, only a logit above kFewRange asks for more.
        const bool zero = set == row_bits && !moved;
        uint32_t bits = 0;
        float top = x[0];
#pragma unroll
        for (int n = 1; n < R; ++n)
            top = fmaxf(top, x[n]);
        if (!zero || top * c > kFewRange) {
#pragma unroll
            for (int n = 0; n < R; ++n) {
                const float z = x[n] * c;
                const bool unset = m[n] == kNegInf, large = z > (unset ? 0.f : m[n]) + kFewRange;
                if (z >= -kFewRange)
                    bits |= 1u << n;
                if (large || (unset && z < -kFewRange && z > kNegInf))
                    bits |= 0x10000u << n;
            }
        }
        bits = __reduce_or_sync(0xffffffffu, bits);
        if (lane == 0)
            sm.rows[t][ct.tiles & 1][wq] = bits;
        float w[R];
        few_exp(x, c, m, !moved, w);
        if (!group_sync())
            return false;
        {
            const volatile uint32_t *all = sm.rows[t][ct.tiles & 1];
            bits = all[0] | all[1] | all[2] | all[3];
        }
        if (kk > 0) {
            // the previous tile's product has read P and landed in O^T
            if (!warp_wait(bar(sm.pv_done[t][0]), ct.pv & 1, cx.wc, W_O_FULL))
                return false;
            ++ct.pv;
            ptx::tc_fence_after();
        }
        if (bits || inf.n_parts == 0) {
            // columns past the item's rows may hold anything and ask for nothing
            const uint32_t ask = (bits >> 16) & row_bits;
            if (ask) {
#pragma unroll
                for (int n = 0; n < R; ++n) {
                    const int mx = __reduce_max_sync(0xffffffffu, ordered(x[n] * c));
                    if (lane == n)
                        sm.red[t][wq][n] = unordered(mx);
                }
                if (!group_sync())
                    return false;
            }
            float alpha[R];
#pragma unroll
            for (int n = 0; n < R; ++n) {
                float m_new = !(set >> n & 1u) && (bits >> n & 1u) ? 0.f : m[n];
                if (ask >> n & 1u) {
                    const volatile float *red = &sm.red[t][0][n];
                    m_new = fmaxf(fmaxf(fmaxf(red[0], red[kFewRows]), fmaxf(red[2 * kFewRows], red[3 * kFewRows])),
                                  m[n]);
                    moved = true;
                }
                alpha[n] = m[n] == kNegInf ? 0.f : ptx::ex2(m[n] - m_new);
                m[n] = m_new;
            }
            set |= (bits | bits >> 16) & row_bits;
            if (ask) {
                if (kk > 0) {
                    uint32_t o[2 * R];
                    few_load_o<R>(tO, o);
#pragma unroll
                    for (int n = 0; n < R; ++n) { // a row without a key so far holds zeros
                        o[n] = __float_as_uint(__uint_as_float(o[n]) * alpha[n]);
                        o[R + n] = __float_as_uint(__uint_as_float(o[R + n]) * alpha[n]);
                        l[n] *= alpha[n];
                    }
                    if constexpr (R == 8)
                        ptx::tmem_st16(tO, o);
                    else
                        ptx::tmem_st32(tO, o);
                    ptx::tmem_wait_st();
                }
                few_exp(x, c, m, false, w);
            }
        }
        // the key's row of P: R rounded weights, then R rests
        uint32_t hi[R / 2], lo[R / 2];
#pragma unroll
        for (int n = 0; n < R; n += 2) {
            hi[n / 2] = ptx::pack_bf16(w[n], w[n + 1]);
            lo[n / 2] = ptx::pack_bf16(w[n] - __uint_as_float(hi[n / 2] << 16),
                                       w[n + 1] - __uint_as_float(hi[n / 2] & 0xffff0000u));
        }
#pragma unroll
        for (int u = 0; u < R / 8; ++u) {
            pdst[u ^ sw] = make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]);
            pdst[(R / 8 + u) ^ sw] = make_uint4(lo[4 * u], lo[4 * u + 1], lo[4 * u + 2], lo[4 * u + 3]);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(sm.p_full[t][0]));
#pragma unroll
        for (int n = 0; n < R; n += 2)
            ptx::add2(l[n], l[n + 1], w[n], w[n + 1]);
    }
    if (n_mine) {
        if (!warp_wait(bar(sm.pv_done[t][0]), ct.pv & 1, cx.wc, W_O_FULL))
            return false;
        ++ct.pv;
        ptx::tc_fence_after();
    }
    if (inf.n_parts == 0) // the warm-up
        return true;
    // ---- the slot's sums over the warp, halved at each exchange until lane i
    // holds row i mod R
#pragma unroll
    for (int h = R / 2; h; h >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i)
            l[i] = (up ? l[i + h] : l[i]) + __shfl_xor_sync(0xffffffffu, up ? l[i] : l[i + h], h);
    }
#pragma unroll
    for (int d = R; d < 32; d *= 2)
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
    float o[R];
    if (n_mine) {
        uint32_t raw[2 * R];
        few_load_o<R>(tO, raw);
#pragma unroll
        for (int n = 0; n < R; ++n)
            o[n] = __uint_as_float(raw[n]) + __uint_as_float(raw[R + n]);
    } else {
#pragma unroll
        for (int n = 0; n < R; ++n)
            o[n] = 0.f;
    }
    // lane = dimension; at D = 64 the upper 64 lanes repeat the lower ones and
    // take the odd rows
    const int dim = D == 128 ? r : r & 63;
    if (inf.n_parts > 1) {
        float *mine = partial<D>(p, inf.cta, inf.mine, t), *sums = mine + kFewRows * 128;
#pragma unroll
        for (int n = 0; n < R; ++n) {
            if (n < rows && (D == 128 || (n & 1) == r >> 6))
                mine[n * 128 + dim] = o[n];
            if (r == n)
                sums[n] = m[n];
        }
        if (lane < R)
            sums[kFewRows + wq * kFewRows + lane] = l[0];
        return true;
    }
    if (!n_mine && !group_sync()) // the last item's sums have been read
        return false;
    if (lane < R)
        sm.red[t][wq][lane] = l[0];
    if (!group_sync())
        return false;
    // a row's sum per lane, so that the reciprocals and logarithms are taken at once
    const volatile float *red = sm.red[t][0] + (lane & (R - 1));
    const float sum = red[0] + red[kFewRows] + red[2 * kFewRows] + red[3 * kFewRows];
    const float inv = sum == 0.f ? 0.f : ptx::rcp_approx(sum);
#pragma unroll
    for (int n = 0; n < R; ++n) {
        const float norm = __shfl_sync(0xffffffffu, inv, n);
        if (n >= rows || (D == 64 && (n & 1) != r >> 6))
            continue;
        const int s = fast_div(n, p.div_g);
        const int64_t tok = inf.t0 + s, head = (inf.kvh + t) * p.G + n - s * p.G;
        p.out[tok * p.o_st + head * p.o_sh + dim] = __float2bfloat16(o[n] * norm);
    }
    if (r < rows) {
        float ref = m[0];
#pragma unroll
        for (int n = 1; n < R; ++n)
            ref = r == n ? m[n] : ref;
        const int s = fast_div(r, p.div_g);
        join_lse(p, inf.t0 + s, (inf.kvh + t) * p.G + r - s * p.G, ref, sum);
    }
    return true;
}

template <int MOD, int D>
__device__ void few_softmax(const FewCtx<D, false> &cx, const ChunkParams &p, int t)
{
    FewSmem<D, false> &sm = *cx.sm;
    FewState ct{0u, 0u, 0u, 0u};
    for (uint32_t item = 0;; ++item) {
        if (!warp_wait(bar(sm.info_full[item % kInfo]), (item / kInfo) & 1, cx.wc, W_INFO_FULL))
            return;
        const FewItem &inf = sm.info[item % kInfo];
        if (inf.stop)
            return;
        // an odd head's item has no second slot; half the rows, half the work
        if (t < inf.heads && !(inf.rows <= 8 ? few_item<MOD, D, 8>(cx, p, inf, t, ct)
                                             : few_item<MOD, D, 16>(cx, p, inf, t, ct)))
            return;
        __syncwarp();
        if (ptx::lane_id() == 0)
            ptx::mbar_arrive(bar(sm.info_empty[item % kInfo]));
    }
}

// ------------------------------------------------------------------ softmax, 8 bits
//
// A thread has keys r (and, of a tile of 256, 128 + r).  One reference a row, ref, for the
// weights times V's scale, P = 2^(z + lv - ref) with lv = kFewTop + log2 s, and one for the row's
// sum, of 2^(z - m) with m = ref - gap: scales may be 2^200 apart (a block of zeros has 2^-100), so
// neither exponential can be had from the other.  The references make the largest P of a tile
// 2^kFewTop and the largest weight 1 when they are set, and are set again where one would pass
// 2^kFewMost or 2^kFewSumMost: until then the slot's warps only agree, once a tile, that none does.
// (The second exponentials take 64 tokens on 512 to 8192 keys from 68 to 69 us.  A function of its own for
// scales far apart took 75, two copies of the code for P 79: what this loop costs is its instructions'
// fetch.)
//
// P is rounded to f16, 11 bits down to 2^-26 of the row's largest and steps of 2^-36 of it
// below, and goes as three e5m2 terms of 3 bits and a sign each, 16 times apart, which hold
// f16 exactly.  (In two e4m3 terms, 9 bits from 2^2 on and steps of 2^-13, a row that has most of its
// weight on one key lost the others': relative errors of 0.1 to 0.5 at 8192 to 32768 keys.)

constexpr float kFewTop = 12.f, kFewMost = 14.8f; // rounded to e5m2, 2^14.8 times 2^-3 times 16 stays in range
constexpr float kFewSumMost = 60.f;
constexpr int kFewTerms = 3;

struct FewState8 {
    uint32_t s, group, tiles; // phases of s_full, group; tiles so far
    uint32_t loaded;          // tiles of the CTA before this item
};

// Four numbers to f16, and those to three e5m2 terms (the upper bytes of f16 numbers): a term
// is what is left, rounded; what that leaves is exact, and is multiplied by 16.
__device__ __forceinline__ void split_p(const float (&e)[4], uint32_t &t0, uint32_t &t1, uint32_t &t2)
{
    uint32_t a = ptx::pack_f16(e[0], e[1]), b = ptx::pack_f16(e[2], e[3]);
    auto rounded = [](uint32_t x) { return (x + 0x00800080u) & 0xff00ff00u; };
    auto rest = [](uint32_t x, uint32_t t) {
        const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&t)),
                                  __half2half2(__ushort_as_half(0x4c00))); // 16
        return *reinterpret_cast<const uint32_t *>(&r);
    };
    uint32_t ra = rounded(a), rb = rounded(b);
    t0 = __byte_perm(ra, rb, 0x7531);
    a = rest(a, ra), b = rest(b, rb);
    ra = rounded(a), rb = rounded(b);
    t1 = __byte_perm(ra, rb, 0x7531);
    t2 = __byte_perm(rounded(rest(a, ra)), rounded(rest(b, rb)), 0x7531);
}

// A key's row of P and its part of the sums: d = log2 of P; d - lv + gap that of the weight.
template <int R>
__device__ __forceinline__ void few_p8(const float (&d)[R], float lv, uint32_t gap, float (&sum)[R],
                                       uint32_t (&p)[kFewTerms][R / 4])
{
#pragma unroll
    for (int n = 0; n < R; n += 4) {
        float e[4], z[4];
        ptx::load_shared_v4(gap + 4 * n, z);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            ptx::add2(z[i], z[i + 1], -lv, -lv);
            ptx::add2(z[i], z[i + 1], d[n + i], d[n + i + 1]);
            e[i] = ptx::ex2(d[n + i]);
            e[i + 1] = ptx::ex2(d[n + i + 1]);
            ptx::add2(sum[n + i], sum[n + i + 1], ptx::ex2(z[i]), ptx::ex2(z[i + 1]));
        }
        split_p(e, p[0][n / 4], p[1][n / 4], p[2][n / 4]);
    }
}

// 16 columns of O^T at a time, where column c is term c / R of row c % R.
template <int R>
constexpr int kFewColumns = (kFewTerms * R + 15) / 16;

// One item of at most R rows.  False when a wait ran out.
template <int MOD, int D, int R>
__device__ __forceinline__ bool few_item_fp8(const FewCtx<D, true> &cx, const ChunkParams &p, const FewItem &inf, int t,
                                             FewState8 &ct)
{
    using C = FewCfg<D, true>;
    constexpr int kBN = C::kBN, kSub = C::kSub;
    FewSmem<D, true> &sm = *cx.sm;
    const int r = threadIdx.x & 127;
    const int wq = (threadIdx.x >> 5) & 3, lane = static_cast<int>(ptx::lane_id());
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = cx.tmem + lanes + C::kColS + C::kStride * t;
    const uint32_t tO = cx.tmem + lanes + C::kColO + C::kStrideO * t;
    const uint32_t b_group = bar(sm.group[t]);
    ScoreMod smod;
    smod.qk_log2 = p.qk_log2;
    smod.softcap_in = p.softcap_in;
    smod.softcap_out = p.softcap_out;
    smod.alibi_c = smod.scale = smod.b = smod.h = 0.f;
    auto group_wait = [&]() { return warp_wait(b_group, ct.group++ & 1, cx.wc, W_JOIN); };
    const FewTiles f = few_tiles(inf, t);
    const int n_mine = f.hi > f.first ? (f.hi - f.first + f.step - 1) / f.step : 0;
    const int rows = inf.rows, pos0 = inf.pos0;
    int full_lo, full_hi, unused;
    {
        const int last = pos0 + fast_div(rows - 1, p.div_g);
        key_range(p, inf.L, last, last, full_lo, unused);
        key_range(p, inf.L, pos0, pos0, unused, full_hi);
    }
    float ref[R], l[R], q_factor[R];
#pragma unroll
    for (int n = 0; n < R; ++n) {
        const int s = fast_div(n, p.div_g);
        l[n] = 0.f;
        ref[n] = n < rows ? 0.f : 1e30f; // columns past the rows ask for nothing
        q_factor[n] = n < rows && inf.n_parts
                          ? __ldcg(p.q_scale + static_cast<int64_t>(inf.t0 + s) * p.Hq + (inf.kvh + t) * p.G + n - s * p.G) *
                                (MOD == MOD_NONE ? p.qk_log2 : 1.f)
                          : 0.f;
    }
    uint32_t unset = (1u << rows) - 1; // rows without references, which count as 0
    float gap_most = 0.f;      // the largest gap
    volatile float *const gap = sm.sums.gap[t][wq];
    const uint32_t gap_at = ptx::smem_u32(sm.sums.gap[t][wq]);
    __syncwarp();
    if (lane < R)
        gap[lane] = 0.f;
    __syncwarp();
    for (int kk = 0; kk < n_mine; ++kk) {
        if (!warp_wait(bar(sm.s_full[t]), ct.s & 1, cx.wc, W_S_FULL))
            return false;
        ++ct.s;
        const uint32_t buf = ct.tiles % C::kPBufs, buf_phase = (ct.tiles / C::kPBufs) & 1; // of P
        const uint32_t ring = (ct.loaded + static_cast<uint32_t>(f.first + kk * f.step - inf.u_lo)) % kScaleRing;
        volatile uint32_t *const flags = &sm.large[t][ct.tiles & 3];
        const int j0 = ((f.first + kk * f.step) >> inf.shift) * kBN;
        ++ct.tiles;
        ptx::tc_fence_after();
        uint32_t raw[kSub][R];
        float key_k[kSub], log_v[kSub];
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
            if constexpr (R == 4)
                ptx::tmem_ld4(tS + sub * C::kSubS, raw[sub]);
            else if constexpr (R == 8)
                ptx::tmem_ld8(tS + sub * C::kSubS, raw[sub]);
            else
                ptx::tmem_ld16(tS + sub * C::kSubS, raw[sub]);
            key_k[sub] = *const_cast<const volatile float *>(&sm.scales.k[ring][sub * 8 + (r >> 4)]);
            log_v[sub] = *const_cast<const volatile float *>(&sm.scales.v[ring][sub * 8 + (r >> 4)]);
        }
        ptx::tmem_wait_ld();
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub)
            ptx::reg_fence<R>(raw[sub]);
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(sm.s_free[t]));
        // ---- log2 of P, relative to the references as they are
        float d[kSub][R];
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
            log_v[sub] = fmaxf(ptx::lg2(log_v[sub]), kLeastLog) + kFewTop;
            float (&x)[R] = d[sub];
            if constexpr (MOD == MOD_NONE) {
#pragma unroll
                for (int n = 0; n < R; n += 2) {
                    float a0, a1;
                    ptx::fma2(a0, a1, q_factor[n], q_factor[n + 1], key_k[sub], key_k[sub], 0.f, 0.f);
                    ptx::fma2(x[n], x[n + 1], __uint_as_float(raw[sub][n]), __uint_as_float(raw[sub][n + 1]), a0, a1,
                              log_v[sub] - ref[n], log_v[sub] - ref[n + 1]);
                }
            } else {
#pragma unroll
                for (int n = 0; n < R; ++n)
                    x[n] = __uint_as_float(raw[sub][n]) * (q_factor[n] * key_k[sub]);
                apply_score_mod<MOD, R>(x, smod, 0, j0);
#pragma unroll
                for (int n = 0; n < R; ++n)
                    x[n] += log_v[sub] - ref[n];
            }
        }
        if (!(j0 >= full_lo && j0 + kBN <= full_hi)) {
#pragma unroll
            for (int n = 0; n < R; ++n) {
                int lo, hi;
                const int pos = pos0 + fast_div(n, p.div_g);
                key_range(p, inf.L, pos, pos, lo, hi);
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub) {
                    const int key = j0 + sub * 128 + r;
                    if (key < lo || key >= hi)
                        d[sub][n] = kNegInf;
                }
            }
        }
        // does a key ask for a new reference? (at the most)
        bool more = false;
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
            float most = d[sub][0];
#pragma unroll
            for (int n = 1; n < R; ++n)
                most = fmaxf(most, d[sub][n]);
            more |= most > (unset ? kNegInf : kFewMost) || most - log_v[sub] + gap_most > kFewSumMost;
        }
        if (__any_sync(0xffffffffu, more) && lane == 0)
            *flags = 1;
        ptx::mbar_arrive(b_group);
        // ---- P, as if no row did, and again if one does
        float sum[R];
        uint32_t pt[kSub][kFewTerms][R / 4];
#pragma unroll 1
        for (int pass = 0;; ++pass) {
#pragma unroll
            for (int n = 0; n < R; ++n)
                sum[n] = l[n];
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub)
                few_p8<R>(d[sub], log_v[sub], gap_at, sum, pt[sub]);
            if (pass)
                break;
            if (!group_wait())
                return false;
            const bool large = *flags;
            // the word of the next tile but one: every warp has read what it held
            if (r == 0)
                sm.large[t][(ct.tiles + 1) & 3] = 0;
            if (!(large || inf.n_parts == 0))
                break;
            // the largest of each row, over the slot's warps
#pragma unroll
            for (int n = 0; n < R; ++n) {
                float top = d[0][n];
                if constexpr (kSub == 2)
                    top = fmaxf(top, d[1][n]);
                const int mx = __reduce_max_sync(0xffffffffu, ordered(top));
                top = d[0][n] - log_v[0];
                if constexpr (kSub == 2)
                    top = fmaxf(top, d[1][n] - log_v[1]);
                const int mz = __reduce_max_sync(0xffffffffu, ordered(top));
                if (lane == n) {
                    sm.red[t][wq][n] = unordered(mx);
                    sm.sums.most[t][wq][n] = unordered(mz);
                }
            }
            ptx::mbar_arrive(b_group);
            if (!group_wait())
                return false;
            // a row per lane: how far its references move
            auto over_warps = [&](const volatile float *m) {
                return fmaxf(fmaxf(m[0], m[kFewRows]), fmaxf(m[2 * kFewRows], m[3 * kFewRows]));
            };
            const int row = lane & (R - 1);
            const float own_gap = gap[row];
            float row_up = over_warps(&sm.red[t][0][row]) - kFewTop, row_up_m = over_warps(&sm.sums.most[t][0][row]) + own_gap;
            const bool first = unset >> row & 1u;
            const bool moves = row < rows && (first ? row_up > kNegInf : row_up > kFewMost - kFewTop || row_up_m > kFewSumMost);
            // (one that is set may move for the other's sake)
            row_up = !moves ? 0.f : first ? row_up : fmaxf(row_up, 0.f);
            row_up_m = !moves ? 0.f : first ? row_up_m : fmaxf(row_up_m, 0.f);
            const float row_beta = moves && first ? 0.f : ptx::ex2(-row_up), row_beta_l = moves && first ? 0.f : ptx::ex2(-row_up_m);
            const float row_gap = own_gap + row_up - row_up_m;
            __syncwarp();
            if (lane < R)
                gap[lane] = row_gap;
            unset &= ~__ballot_sync(0xffffffffu, moves);
            gap_most = unordered(__reduce_max_sync(0xffffffffu, ordered(row < rows && !(unset >> row & 1u) ? row_gap : 0.f)));
            __syncwarp();
            float beta[R];
#pragma unroll
            for (int n = 0; n < R; ++n) {
                const float up = __shfl_sync(0xffffffffu, row_up, n);
                beta[n] = __shfl_sync(0xffffffffu, row_beta, n);
                ref[n] += up;
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub)
                    d[sub][n] -= up;
                l[n] *= __shfl_sync(0xffffffffu, row_beta_l, n);
            }
            if (kk > 0) {
                const uint32_t last = ct.tiles - 2; // the tile before, its product done
                if (!warp_wait(bar(sm.pv_done[t][last % C::kPBufs]), (last / C::kPBufs) & 1, cx.wc, W_O_FULL))
                    return false;
                ptx::tc_fence_after();
#pragma unroll
                for (int i = 0; i < kFewColumns<R>; ++i) {
                    uint32_t o[16];
                    ptx::tmem_ld16(tO + 16 * i, o);
                    ptx::tmem_wait_ld();
                    ptx::reg_fence<16>(o);
#pragma unroll
                    for (int c = 0; c < 16; ++c) // a row without a key so far holds zeros
                        o[c] = __float_as_uint(__uint_as_float(o[c]) * beta[(16 * i + c) % R]);
                    ptx::tmem_st16(tO + 16 * i, o);
                }
                ptx::tmem_wait_st();
            }
        }
#pragma unroll
        for (int n = 0; n < R; ++n)
            l[n] = sum[n];
        if (kk >= C::kPBufs) {
            // the product of the buffer's last tile has read it
            if (!warp_wait(bar(sm.pv_done[t][buf]), buf_phase ^ 1, cx.wc, W_O_FULL))
                return false;
        }
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
            // 16 bytes of a key beside those of the next, the key's others kBN * 16 further
            uint4 *const pdst = reinterpret_cast<uint4 *>(sm.p[t][buf]) + sub * 128 + r;
            const uint32_t(&w)[kFewTerms][R / 4] = pt[sub];
            if constexpr (R == 4) {
                pdst[0] = make_uint4(w[0][0], w[1][0], w[2][0], 0);
            } else if constexpr (R == 8) {
                pdst[0] = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
                pdst[kBN] = make_uint4(w[2][0], w[2][1], 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < kFewTerms; ++i)
                    pdst[i * kBN] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(sm.p_full[t][buf]));
    }
    if (n_mine) {
        const uint32_t last = ct.tiles - 1;
        if (!warp_wait(bar(sm.pv_done[t][last % C::kPBufs]), (last / C::kPBufs) & 1, cx.wc, W_O_FULL))
            return false;
        ptx::tc_fence_after();
    }
    if (inf.n_parts == 0) // the warm-up
        return true;
    // ---- the slot's sums over the warp, halved at each exchange until lane i
    // holds row i mod R
#pragma unroll
    for (int h = R / 2; h; h >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i)
            l[i] = (up ? l[i + h] : l[i]) + __shfl_xor_sync(0xffffffffu, up ? l[i] : l[i + h], h);
    }
#pragma unroll
    for (int d = R; d < 32; d *= 2)
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
    float o[R];
#pragma unroll
    for (int n = 0; n < R; ++n)
        o[n] = 0.f;
    if (n_mine) {
        constexpr float kTerm[] = {0x1p-12f, 0x1p-16f, 0x1p-20f}; // of 2^kFewTop, 16 apart
#pragma unroll
        for (int i = 0; i < kFewColumns<R>; ++i) {
            uint32_t raw[16];
            ptx::tmem_ld16(tO + 16 * i, raw);
            ptx::tmem_wait_ld();
            ptx::reg_fence<16>(raw);
#pragma unroll
            for (int c = 16 * i; c < min(16 * i + 16, kFewTerms * R); ++c)
                o[c % R] = fmaf(__uint_as_float(raw[c % 16]), kTerm[c / R], o[c % R]);
        }
    }
    // lane i's row, i mod R: m, and log2 of O's unit relative to 2^m
    const int row = lane & (R - 1);
    const float unit = gap[row];
    float m = ref[0];
#pragma unroll
    for (int n = 1; n < R; ++n)
        m = row == n ? ref[n] : m;
    m = unset >> row & 1u ? kNegInf : m - unit; // or no key
    // lane = dimension; at D = 64 the upper 64 lanes repeat the lower ones and
    // take the odd rows
    const int dim = D == 128 ? r : r & 63;
    if (inf.n_parts > 1) {
        float *mine = partial<D>(p, inf.cta, inf.mine, t), *sums = mine + kFewRows * 128;
#pragma unroll
        for (int n = 0; n < R; ++n)
            if (n < rows && (D == 128 || (n & 1) == r >> 6))
                mine[n * 128 + dim] = o[n];
        if (lane < R) {
            sums[kFewRows + wq * kFewRows + lane] = l[0];
            if (wq == 0) {
                sums[lane] = m;
                sums[5 * kFewRows + lane] = unit;
            }
        }
        return true;
    }
    auto group_sync = [&]() {
        ptx::mbar_arrive(b_group);
        return group_wait();
    };
    if (!n_mine && !group_sync()) // the last item's sums have been read
        return false;
    if (lane < R)
        sm.red[t][wq][lane] = l[0];
    if (!group_sync())
        return false;
    // a row's sum per lane, so that the reciprocals and logarithms are taken at once
    const volatile float *red = sm.red[t][0] + row;
    const float sum = red[0] + red[kFewRows] + red[2 * kFewRows] + red[3 * kFewRows];
    const float inv = few_norm(sum, unit);
#pragma unroll
    for (int n = 0; n < R; ++n) {
        const float norm = __shfl_sync(0xffffffffu, inv, n);
        if (n >= rows || (D == 64 && (n & 1) != r >> 6))
            continue;
        const int s = fast_div(n, p.div_g);
        const int64_t tok = inf.t0 + s, head = (inf.kvh + t) * p.G + n - s * p.G;
        p.out[tok * p.o_st + head * p.o_sh + dim] = __float2bfloat16(o[n] * norm);
    }
    if (r < rows) {
        const int s = fast_div(r, p.div_g);
        join_lse(p, inf.t0 + s, (inf.kvh + t) * p.G + r - s * p.G, m, sum);
    }
    return true;
}

template <int MOD, int D>
__device__ void few_softmax_fp8(const FewCtx<D, true> &cx, const ChunkParams &p, int t)
{
    FewSmem<D, true> &sm = *cx.sm;
    FewState8 ct{0u, 0u, 0u, 0u};
    for (uint32_t item = 0;; ++item) {
        if (!warp_wait(bar(sm.info_full[item % kInfo]), (item / kInfo) & 1, cx.wc, W_INFO_FULL))
            return;
        const FewItem &inf = sm.info[item % kInfo];
        if (inf.stop)
            return;
        // an odd head's item has no second slot; half the rows, half the work
        if (t < inf.heads && !(inf.rows <= 4   ? few_item_fp8<MOD, D, 4>(cx, p, inf, t, ct)
                               : inf.rows <= 8 ? few_item_fp8<MOD, D, 8>(cx, p, inf, t, ct)
                                               : few_item_fp8<MOD, D, 16>(cx, p, inf, t, ct)))
            return;
        ct.loaded += inf.u_hi - inf.u_lo;
        __syncwarp();
        if (ptx::lane_id() == 0)
            ptx::mbar_arrive(bar(sm.info_empty[item % kInfo]));
    }
}

// The kernel of the few rows (see chunk_kernel for what runs beside it).
template <int MOD, int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_few_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkParams p)
{
    using C = FewCfg<D, F8>;
    extern __shared__ uint8_t smem_raw[];
    FewSmem<D, F8> *sm = reinterpret_cast<FewSmem<D, F8> *>(smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5;
    FewCtx<D, F8> cx;
    cx.part = part_of(p);
    if (idle_second(p, 1, cx.part))
        return;

    if (threadIdx.x == 0) {
        ptx::prefetch_tensormap(&maps.few_q);
        ptx::prefetch_tensormap(&maps.few_k);
        ptx::prefetch_tensormap(&maps.few_v);
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar(sm->q_full[b]), 1);
            ptx::mbar_init(bar(sm->q_empty[b]), 1);
        }
        for (int b = 0; b < kInfo; ++b) {
            ptx::mbar_init(bar(sm->info_full[b]), 1);
            ptx::mbar_init(bar(sm->info_empty[b]), 11); // all but the producer
        }
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(bar(sm->k_full[s]), F8 ? 1 + kScaleArrivals : 1);
            ptx::mbar_init(bar(sm->k_empty[s]), F8 ? 2 : 1); // S's; in 8 bits O^T's, too
            if constexpr (!F8) {
                ptx::mbar_init(bar(sm->v_full[s]), 1);
                ptx::mbar_init(bar(sm->v_empty[s]), few_split_loads<F8>(p) ? 1 : 2); // the warps that issue O^T
            }
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(bar(sm->s_full[t]), 1);
            ptx::mbar_init(bar(sm->s_free[t]), 128);
            for (int b = 0; b < C::kPBufs; ++b) {
                ptx::mbar_init(bar(sm->p_full[t][b]), 128);
                ptx::mbar_init(bar(sm->pv_done[t][b]), 1);
            }
            ptx::mbar_init(bar(sm->group[t]), 128);
        }
        for (int b = 0; b < 3; ++b)
            ptx::mbar_init(bar(sm->final_bar[b]), 1);
        for (int b = 0; b < 8; ++b)
            sm->large[b >> 2][b & 3] = 0;
        sm->abort_flag = 0;
        ptx::fence_mbarrier_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&sm->tmem_base), C::kColumns);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();

    cx.sm = sm;
    cx.tmem = sm->tmem_base;
    cx.wc = wait_ctl(p, &sm->abort_flag);
    if (warp >= 4) {
        tell_second(p, cx.part);
        if constexpr (F8)
            few_softmax_fp8<MOD, D>(cx, p, (warp >> 2) - 1);
        else
            few_softmax<MOD, D>(cx, p, (warp >> 2) - 1);
        ptx::tc_fence_before();
        ptx::named_barrier_sync(1, kThreads);
    } else {
        if (warp == 0) {
            if constexpr (F8)
                few_loader_fp8(cx, p, &maps.few_q, &maps.few_k, &maps.few_v);
            else
                few_producer(cx, p, &maps.few_q, &maps.few_k, &maps.few_v);
        } else if (warp == 1)
            few_s_role(cx);
        else if (!F8 && !few_split_loads<F8>(p))
            few_pv_role(cx, warp - 2, warp - 2);
        else if (warp == 2)
            few_pv_role(cx, 0, 1);
        else if constexpr (F8)
            few_walker_fp8(cx, p);
        else
            few_v_producer(cx, p, &maps.few_v);
        ptx::tc_fence_before();
        ptx::named_barrier_sync(1, kThreads);
        if (warp == 1) {
            ptx::tc_fence_after();
            ptx::tmem_dealloc(cx.tmem, C::kColumns);
        }
        ptx::wait_dependency(); // see chunk_plan.cuh
    }
}

} // namespace
} // namespace fl
