// chunk_blocks.cuh -- the kernels of fwd_chunk.cu and fwd_chunk_fp8.cu:
// attention of ragged chunks of new tokens over the cache that holds them
// (serving: prompts, parts of prompts and single tokens in one call), paged or
// contiguous, in bf16 or 8 bits (F8); D = 64 or 128.
//
// Mathematics: the online softmax of softmax_tile.cuh; rows whose keys are
// split over several SMs leave partial (m, l, O) and are joined by
//     M = max m_i,  O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
//
// Work.  The query rows of a (request, KV head) are its tokens times the G
// query heads of the group, token by token, so that even one token of a
// grouped head shares every key load among its heads.  Up to 16 rows are "few
// rows" (chunk_few.cuh); more make row blocks of TQ = 128 / G tokens, which
// fill the 128 rows of an MMA, and are this file's.  An item is two such blocks
// (or the last one) of one request and KV head, against the key tiles any of
// its rows sees.  Lengths live on the device, so a one-block planning kernel
// (chunk_plan.cuh) lists the items of both kinds with a running sum of their
// cost, shares the SMs between the lists and cuts each list's sum into equal
// parts, one per CTA: CTAs start and stop in the middle of an item's keys,
// wherever the cut falls, so a single long conversation spreads over the GPU as
// evenly as a full batch, and a batch needs no heuristics for the number of
// splits.  At most the first and last item of a CTA are shared; these leave
// partials in the workspace, which a kernel of their own joins in the order
// of the keys.  The launches overlap (programmatic dependent launch).
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
// (short chunks) gives both slots the same rows and every second key tile, and
// the slots' results are joined in the epilogue, each warpgroup reading both
// accumulators from TMEM for half of the columns.  Warps that hold no row of
// the item skip the arithmetic.
//
// K/V tiles are 112 keys at D = 64 and 64 at D = 128 (TMEM budget of the
// standard kernel), loaded as boxes of 16 keys: the largest that divides the
// tile and every page size.  Keys no row may see never reach the sums: logits
// are replaced by -inf, and as 0 * NaN is not 0, the S warp zeroes those rows
// of V in shared memory (only in tiles at the ends of the cache or window).
//
// Bound by no one pipe but by the chain of dependent instructions in each of
// the two softmax warps a scheduler has: the last 4096 tokens of 16384, 32 heads
// over 8 of 64, take 457 us, 1050 TFLOP/s, with the tensor pipe 50% active,
// special functions 44% and 56% of the issue slots used; 16 heads over 2 of 128
// 410 us, 1170 TFLOP/s (1.05 us a pair of blocks and tile).  An
// item costs 2 to 3 us more (its last product, O out of TMEM, its rows to
// memory), which is what short windows and chunks pay.
//
// A cache in 8 bits: S as in chunk_few.cuh, K's codes against Q's two terms.  For
// O, warps 2 and 3 turn V's codes into f16 (exact) in shared memory while the
// softmax of the next tile runs, and P is f16 with V's scale in its exponent, one for 16
// keys, relative to the largest product of weight and scale of the row (softmax_compute_p_scaled).
// V's codes straight into the product want P in 8 bits, in three terms for as much: three times the
// rows of the 128 an MMA has.  Converted by the softmax's own warps the long prompt above took 1.6
// times as long.
// It takes 583 us, 825 TFLOP/s: the conversion and the factors are 15% more instructions (issue
// 50%, tensor 32%, special functions 34%); at D = 128 433 us, 1110 TFLOP/s.  Windows of 1024 keys,
// 4023 tokens, 16 heads over 2 of 128: 69 us, 64 in bf16.
#pragma once

#include <cuda_bf16.h>
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "chunk_few.cuh"
#include "chunk_plan.cuh"
#include "common.cuh"
#include "fp8.cuh"
#include "launch.h"
#include "softmax_tile.cuh"

namespace fl {
namespace {

constexpr int kBox = 16; // keys per TMA box

template <int D, bool F8 = false>
struct ChunkCfg {
    static_assert(D == 64 || D == 128, "head dimension");
    static constexpr int kBN = chunk_key_tile(D);
    static constexpr int kStages = D == 128 ? 3 : 4; // of K and V as they are loaded
    static constexpr int kVStages = F8 ? (D == 128 ? 2 : 3) : kStages; // of V in 16 bits
    static constexpr bool kOnes = D <= 64 && !F8; // sum of the rounded P from a ones column block
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kRowBytes = 128;
    static constexpr uint32_t kGroupBytes = 8 * kRowBytes;
    static constexpr uint32_t kQHalf = BM * kRowBytes;
    static constexpr uint32_t kKVHalf = kBN * kRowBytes;
    static constexpr uint32_t kTileBytes = kHalves * kQHalf;
    static constexpr uint32_t kKVBytes = kHalves * kKVHalf;
    static constexpr uint32_t kLoadBytes = F8 ? kBN * D : kKVBytes; // of a tile of K or V as it is loaded
    static constexpr uint32_t kRowSwizzle = F8 && D == 64 ? kSwizzle64B : kSwizzle128B; // of Q and K
    static constexpr uint32_t kRowLen = F8 ? D : kRowBytes;
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
    int n_parts;                 // CTAs that share the item
    int cta;                     // this part among those of both paths
    int mine;                    // its buffer: 1 if the item begins here
};

template <int D, bool F8>
struct __align__(1024) ChunkSmem {
    using C = ChunkCfg<D, F8>;
    uint8_t q[2][2][C::kTileBytes]; // [Q buffer][slot]; in 8 bits two terms
    uint8_t k[C::kStages][C::kLoadBytes];
    uint8_t v[C::kVStages][C::kKVBytes];
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
    // a cache in 8 bits: V as it is loaded, and the stages of what it is converted to
    uint64_t v_full[F8 ? C::kVStages : 1], v_empty[F8 ? C::kVStages : 1];
    std::conditional_t<F8, ScaleRing, char> scales;
    std::conditional_t<F8, TileFactors, char> factors[2][4]; // [slot][its tiles in turn]
    alignas(F8 ? 128 : 4) uint8_t raw_v[F8 ? C::kStages : 1][F8 ? C::kLoadBytes : 4];
};

template <int D, bool F8>
struct KernelCtx {
    ChunkSmem<D, F8> *sm;
    uint32_t tmem;
    int part;
    WaitCtl wc;
};

// ------------------------------------------------------------------ producer

template <int D, bool F8>
__device__ void producer_role(const KernelCtx<D, F8> &cx, const ChunkParams &p, const CUtensorMap *tm_q,
                              const CUtensorMap *tm_k, const CUtensorMap *tm_v)
{
    using C = ChunkCfg<D, F8>;
    constexpr int kBN = C::kBN, kStages = C::kStages, kBoxes = kBN / kBox;
    ChunkSmem<D, F8> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    uint32_t kv_count = 0, item_count = 0;
    bool ok = true;
    ChunkPart me{};
    const int cta = cx.part;
    int e = 0, h = 0, k = 0; // entry, item of it, tile of that
    read_part(p, 0, cta, me, e, h, k);
    if (F8)
        ptx::fence_proxy_async_all(); // Q's terms, which the planning kernel has written
    for (;;) {
        // ---- the next part
        Item it;
        it.stop = 1;
        ChunkEntry en{};
        int k_end = 0;
        while (e < me.n_entries) {
            en = e == me.entry ? me.at : load_plan(p.entries + e);
            const int64_t x0 = en.cum + h * item_cost(p, en);
            if (x0 + static_cast<int64_t>(k) * en.tile_cost >= me.end) {
                e = me.n_entries; // the cut falls before this tile
                break;
            }
            if (k < en.n_tiles) {
                const PartRange r = part_range(x0, en.n_tiles, en.tile_cost, k, me.end, me.total, cta, me.parts);
                k_end = r.k_end;
                it.n_parts = r.n_parts;
                it.mine = r.first == cta ? 1 : 0;
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
            it.cta = me.cta;
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
            // an item whose rows see no key has no tile: one that no slot uses would be
            // released by the P V warps alone, while the S warp may still be zeroing
            // its rows of V
            it.u_hi = max(it.u_lo, max(it.hi[0], it.hi[1]));
        }
        const uint32_t ring = item_count & 1, slot = item_count % kInfo;
        ok = warp_wait(bar(sm.info_empty[slot]), ((item_count / kInfo) & 1) ^ 1, cx.wc, W_INFO_EMPTY);
        if (!ok)
            break;
        if (lane == 0) {
            sm.info[slot] = it;
            ptx::mbar_arrive(bar(sm.info_full[slot])); // release: the fields above first
            if (!it.stop && it.mine && it.n_parts > 1)
                p.joins[me.cta] = ChunkJoin{it.n_parts, it.pair ? JOIN_PAIR : JOIN_HALF, it.kvh,
                                                {it.t0[0], it.t0[1]}, {it.rows[0], it.rows[1]}, 0};
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
            for (int t = 0; t < slots; ++t) {
#pragma unroll
                for (int hf = 0; hf < (F8 ? 0 : C::kHalves); ++hf)
                    ptx::tma_load_4d(ptx::smem_u32(sm.q[ring][t]) + hf * C::kQHalf, tm_q, bar(sm.q_full[ring]),
                                     hf * 64, 0, it.kvh, it.t0[t]);
#pragma unroll
                for (int i = 0; i < (F8 ? 2 : 0); ++i) // the terms
                    ptx::tma_load_4d(ptx::smem_u32(sm.q[ring][t]) + i * (BM * D), tm_q, bar(sm.q_full[ring]), 0, 0,
                                     it.kvh, it.t0[t] + i * p.T);
            }
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
            if constexpr (F8)
                copy_scales<kBoxes>(p, sm.scales, kv_count, bar(sm.kv_full[s]), page, 4, j * kBN, it.key_lo, it.L, it.kvh);
            const int left = it.L - j * kBN;
            const int boxes = left <= 0 ? 0 : min(kBoxes, (left + kBox - 1) / kBox);
            const uint32_t b_full = bar(sm.kv_full[s]);
            if (lane == 0)
                ptx::mbar_arrive_expect_tx(b_full, static_cast<uint32_t>(2 * boxes * kBox) * (F8 ? 1 : 2) * D);
            __syncwarp();
            if (static_cast<int>(lane) < boxes) {
                const int key = j * kBN + static_cast<int>(lane) * kBox;
                const int at = p.page_shift < 0 ? key : key & ((1 << p.page_shift) - 1);
                if constexpr (F8) {
                    ptx::tma_load_4d(ptx::smem_u32(sm.k[s]) + lane * kBox * D, tm_k, b_full, 0, at, it.kvh, page);
                    ptx::tma_load_4d(ptx::smem_u32(sm.raw_v[s]) + lane * kBox * D, tm_v, b_full, 0, at, it.kvh, page);
                }
                const uint32_t off = lane * kBox * C::kRowBytes;
#pragma unroll
                for (int hf = 0; hf < (F8 ? 0 : C::kHalves); ++hf) {
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

template <int MOD, int D, bool F8>
__device__ void s_role(const KernelCtx<D, F8> &cx)
{
    using C = ChunkCfg<D, F8>;
    constexpr int kBN = C::kBN, kStages = C::kStages;
    ChunkSmem<D, F8> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    constexpr uint32_t idesc_qk = F8 ? umma_idesc_e4m3(BM, kBN) : umma_idesc_bf16(BM, kBN, false);
    constexpr uint64_t kHiK = umma_desc_hi(16, 8 * C::kRowLen, C::kRowSwizzle); // Q, K: K-major
    constexpr uint32_t kTileLo = C::kTileBytes >> 4, kKVLo = C::kLoadBytes >> 4;
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
            float scale_k = 0.f, scale_v = 0.f;
            if constexpr (F8) if ((lane & 7) < kBN / 16) {
                scale_k = *const_cast<const volatile float *>(&sm.scales.k[idx % kScaleRing][lane & 7]);
                scale_v = *const_cast<const volatile float *>(&sm.scales.v[idx % kScaleRing][lane & 7]);
            }
            // rows of V that no query row sees: zero (their P is 0, but the bytes
            // may be anything); with softcap those of K, too (softcap_scores).  Some slot
            // uses every tile, and its P V, which releases the stage, waits for this
            // warp's S.  Each lane's writes reach the tensor core through its proxy fence, the S
            // issue, s_full, p_full and the P V issue.
            const int j0 = j * kBN;
            const int dead_lo = min(kBN, max(0, key_lo - j0)), dead_hi = min(kBN, max(0, L - j0));
            if ((!F8 || MOD == MOD_SOFTCAP) && (dead_lo > 0 || dead_hi < kBN)) {
                constexpr int kUnits = C::kRowLen / 16;
#pragma unroll
                for (int hf = F8 ? C::kHalves : 0; hf < (MOD == MOD_SOFTCAP ? 2 : 1) * C::kHalves; ++hf) {
                    if (F8 && hf > C::kHalves) // whole rows of K; V's the conversion has zeroed
                        break;
                    uint4 *v = reinterpret_cast<uint4 *>((hf < C::kHalves ? sm.v[stage] : sm.k[stage]) +
                                                         hf % C::kHalves * C::kKVHalf);
                    for (int c = lane; c < dead_lo * kUnits; c += 32)
                        v[c] = make_uint4(0, 0, 0, 0);
                    for (int c = dead_hi * kUnits + lane; c < kBN * kUnits; c += 32)
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
                // four places: with the last tile's S the softmax was done with the one before that
                if constexpr (F8)
                    tile_factors(sm.factors[t][issued[t] & 3], scale_k, scale_v);
                if (issued[t] > 0) {
                    // the softmax has copied the slot's previous S out of TMEM
                    ok = warp_wait(bar(sm.s_free[t]), (issued[t] - 1) & 1, cx.wc, W_S_FULL);
                    if (!ok)
                        break;
                }
                ++issued[t];
                if (F8) {
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(bar(sm.s_full[t])); // release: the factors first
                }
                ptx::tc_fence_after();
                if (lane == 0) {
                    const uint32_t qlo = q_lo0 + (2 * ring + (pair ? t : 0)) * kTileLo;
                    const uint32_t tS = cx.tmem + C::kColS + C::kStrideS * t;
                    if constexpr (F8) { // both terms of Q with the same K
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            ptx::mma_ss_f8(tS, kHiK | (qlo + kk / (D / 32) * (BM * D >> 4) + 2 * (kk % (D / 32))),
                                           kHiK | (klo + 2 * (kk % (D / 32))), idesc_qk, kk > 0 ? 1u : 0u);
                    }
#pragma unroll
                    for (int kk = 0; kk < (F8 ? 0 : D / 16); ++kk) {
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
            if (F8) {
                if (lane == 0)
                    ptx::mma_commit(bar(sm.kv_empty[stage])); // K has been read
                __syncwarp();
            }
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

template <int D, bool F8>
__device__ void pv_role(const KernelCtx<D, F8> &cx, int t)
{
    using C = ChunkCfg<D, F8>;
    constexpr int kBN = C::kBN, kStages = C::kVStages;
    ChunkSmem<D, F8> &sm = *cx.sm;
    const uint32_t lane = ptx::lane_id();
    uint64_t *const full = F8 ? sm.v_full : sm.kv_full, *const empty = F8 ? sm.v_empty : sm.kv_empty;
    constexpr uint32_t idesc_pv = F8 ? umma_idesc_f16(BM, C::kDvExt, true) : umma_idesc_bf16(BM, C::kDvExt, true);
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
        const int first = inf.first[t], hi = inf.hi[t], L = inf.L, key_lo = inf.key_lo;
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(bar(sm.info_empty[slot]));
        if (stop)
            break;
        // 8 bits: this warp's half of V's tile j, the CTA's number i
        auto convert = [&](int j, uint32_t i) {
            if constexpr (F8) {
                const uint32_t from = i % C::kStages, to = i % kStages;
                if (!warp_wait(bar(sm.kv_full[from]), (i / C::kStages) & 1, cx.wc, W_KV_FULL) ||
                    !warp_wait(bar(empty[to]), ((i / kStages) & 1) ^ 1, cx.wc, W_KV_EMPTY))
                    return false;
                const int j0 = j * kBN;
                convert_half<D, kBN>(sm.raw_v[from], sm.v[to], t, min(kBN, max(0, key_lo - j0)),
                                     min(kBN, max(0, L - j0)));
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(bar(full[to]));
                    ptx::mbar_arrive(bar(sm.kv_empty[from]));
                }
            }
            return true;
        };
        // in 8 bits a tile's V is converted when the P V before has been issued
        for (int j = F8 ? u_lo - 1 : u_lo; j < u_hi; ++j) {
            if (j >= u_lo) {
                const uint32_t stage = idx % kStages;
                if (!uses(j, first, hi, step)) {
                    // tile not used by this slot: release it once it has landed
                    ok = warp_wait(bar(full[stage]), (idx / kStages) & 1, cx.wc, W_KV_FULL);
                    if (!ok)
                        break;
                    if (lane == 0)
                        ptx::mbar_arrive(bar(empty[stage]));
                    __syncwarp();
                } else {
                    ok = warp_wait(bar(sm.p_full[t]), pcount & 1, cx.wc, W_P_FULL);
                    if (!ok)
                        break;
                    ++pcount;
                    if (F8) { // S has waited for K alone
                        ok = warp_wait(bar(full[stage]), (idx / kStages) & 1, cx.wc, W_KV_FULL);
                        if (!ok)
                            break;
                    }
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
                        ptx::mma_commit(bar(empty[stage]));
                    }
                    __syncwarp();
                }
                ++idx;
            }
            if (F8 && j + 1 < u_hi) {
                ok = convert(j + 1, idx);
                if (!ok)
                    break;
            }
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
    w.mine = partial<D>(p, inf.cta, inf.mine, t) + r;
    return w;
}

// Epilogue of a pair: the slot's own rows, every column.  An active warp.  (In 8 bits `unit` is O's
// relative to 2^m_ref, and a row of q that is not finite, whose sum is NaN, comes out as NaN.)
template <int D, bool F8>
__device__ __forceinline__ void write_slot(const ChunkParams &p, const Item &inf, int t, int r, uint32_t tO,
                                           const RowState &st, bool any, float unit)
{
    const bool live = r < inf.rows[t], whole = inf.n_parts == 1;
    const RowOut<D> w = row_out<D>(p, inf, t, r);
    const float inv = F8 ? (st.l_round == 0.f ? 0.f : ptx::rcp_approx(st.l_round) * unit) : row_inv_norm(st);
    // an accumulator without a tile, or a row without a key, is not read
    const bool keys = any && (F8 ? !(st.l_round == 0.f) : st.m_ref != kNegInf);
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
                w.mine[(c + i) * 128] = F8 ? __uint_as_float(raw[i]) * unit : __uint_as_float(raw[i]);
        }
    }
    if (whole) {
        if (live && w.lse)
            *w.lse = F8 && st.l != st.l ? st.l : row_lse(st);
        return;
    }
    if (live) {
        w.mine[D * 128] = st.m_ref;
        w.mine[(D + 1) * 128] = st.l;
        w.mine[(D + 2) * 128] = st.l_round;
    }
}

// Epilogue of one row block, after both slots are done: this warpgroup's half
// of the columns from both accumulators.  An active warp.
template <int D, bool F8>
__device__ __forceinline__ void write_joined(const ChunkParams &p, const Item &inf, int t, int r, uint32_t tO,
                                             uint32_t tO_other, uint32_t tX_other, const RowState &st, float unit)
{
    constexpr int H = D / 2;
    const bool live = r < inf.rows[t], whole = inf.n_parts == 1;
    const RowOut<D> w = row_out<D>(p, inf, t, r);
    uint32_t other[4];
    ptx::tmem_ld4(tX_other, other);
    ptx::tmem_wait_ld();
    ptx::reg_fence<4>(other);
    const float m1 = __uint_as_float(other[0]), m = fmaxf(st.m_ref, m1);
    float w0 = st.m_ref == kNegInf ? 0.f : ptx::ex2(st.m_ref - m);
    float w1 = m1 == kNegInf ? 0.f : ptx::ex2(m1 - m);
    const float l = w0 * st.l + w1 * __uint_as_float(other[1]);
    const float lr = w0 * st.l_round + w1 * __uint_as_float(other[2]);
    if constexpr (F8) { // the accumulators' units
        w0 *= unit;
        w1 *= __uint_as_float(other[3]);
    }
    const float inv = (F8 ? lr == 0.f : !(lr > 0.f)) ? 0.f : ptx::rcp_approx(lr);
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
                w.mine[(c + i) * 128] = o[i];
        }
    }
    if (!live)
        return;
    if (whole) {
        if (t == 0 && w.lse)
            *w.lse = (F8 ? l == 0.f : !(l > 0.f)) ? kNegInf : (m + log2f(l)) * kLn2;
    } else {
        w.mine[H * 128] = m;
        w.mine[(H + 1) * 128] = l;
        w.mine[(H + 2) * 128] = lr;
    }
}

// cap tanh(z / cap) as out (1 - 2 / (1 + 2^(in z))) in log2 units, four scores
// to a reciprocal: 1 / a = b c d / (a b c d), with the exponent held to 30, where
// tanh is 1 to the last bit and four factors stay in range.  (NaN stays NaN and
// spreads to the other three, so keys that no row sees are zeroed, as V is.)
// This takes 2.25 special functions a score with the softmax's own in place of 3
// (2048 tokens on 8192 keys, 32 heads over 8 of 64: 265 -> 236 us; 16 over 2 of
// 128: 179 -> 157; two scores to a reciprocal: 248, 164).  They are not the bound:
// the busiest SM of a mixed step uses that pipe 66% of its time; the 112 capped
// scores of a row at D = 64 are held until their maximum is known, and spill.
template <int N>
__device__ __forceinline__ void softcap_scores(float (&x)[N], float in, float out)
{
    const float m2o = -2.f * out;
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        float d[4];
        ptx::fma2(d[0], d[1], x[e], x[e + 1], in, in, 0.f, 0.f);
        ptx::fma2(d[2], d[3], x[e + 2], x[e + 3], in, in, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm("min.NaN.f32 %0, %0, 0f41F00000;" : "+f"(d[i]));
            d[i] = ptx::ex2(d[i]);
        }
        ptx::add2(d[0], d[1], 1.f, 1.f);
        ptx::add2(d[2], d[3], 1.f, 1.f);
        const float a = d[0] * d[1], b = d[2] * d[3], t = ptx::rcp_approx(a * b) * m2o, ta = t * b, tb = t * a;
        ptx::fma2(x[e], x[e + 1], ta, ta, d[1], d[0], out, out);
        ptx::fma2(x[e + 2], x[e + 3], tb, tb, d[3], d[2], out, out);
    }
}

template <int MOD, int D, bool F8>
__device__ void softmax_role(const KernelCtx<D, F8> &cx, const ChunkParams &p, int t)
{
    using C = ChunkCfg<D, F8>;
    constexpr int kBN = C::kBN;
    // the warpgroups of a pair take turns on the exponentials; with softcap at D =
    // 64 they run freely, as in the standard kernel (321 us with turns, 236
    // without; at D = 128 157 and 160)
    constexpr bool kTurns = !F8 && (MOD != MOD_SOFTCAP || D == 128);
    ChunkSmem<D, F8> &sm = *cx.sm;
    const int r = threadIdx.x & 127;            // row of the block = TMEM lane
    const int wq = (threadIdx.x >> 5) & 3;      // warp's quarter of the lanes
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = cx.tmem + lanes + C::kColS + C::kStrideS * t;
    const uint32_t tO = cx.tmem + lanes + C::kColO + C::kStrideO * t;
    const uint32_t tP = cx.tmem + lanes + C::kColP + C::kStrideP * t;
    const uint32_t b_turn_mine = bar(sm.turn[t]), b_turn_other = bar(sm.turn[t ^ 1]);
    uint32_t scount = 0, pvcount = 0, turns = 0, joins = 0;
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
        // rows past the item's (other requests', or whatever Q's buffer held) start with a
        // reference that nothing exceeds: they have no say in when the warp rescales
        RowState st{r < inf.rows[t] ? kNegInf : -kNegInf, 0.f, 0.f};
        float gap = 0.f; // 8 bits: how far the sum's reference is below m_ref
        if (take_turns) // turns of tiles before this slot's
            for (int j = n_mine ? first - inf.u_lo : inf.u_hi - inf.u_lo; j > 0; --j, ++turns) {
                if (!turn_wait())
                    return;
                ptx::mbar_arrive(b_turn_other);
            }
        if (active) {
            const int pos0 = inf.pos0[t], L = inf.L;
            float q_scale = 1.f; // 8 bits: of this row's Q
            if constexpr (F8) {
                const int r_tok = fast_div(r, p.div_g);
                if (r < inf.rows[t])
                    q_scale = __ldcg(p.q_scale + static_cast<int64_t>(inf.t0[t] + r_tok) * p.Hq + inf.kvh * p.G + r - r_tok * p.G);
            }
            const float qk = p.qk_log2 * q_scale, cap_in = p.softcap_in * q_scale;
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
                // 8 bits: the factors of each 16 scores, and of their weights
                float c[F8 ? kBN / 16 : 1], log_v[8];
                if constexpr (F8) {
                    const uint32_t at = ptx::smem_u32(&sm.factors[t][(scount - 1) & 3]);
                    float k[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 4)
                        ptx::load_shared_v4(at + 4 * i, k + i);
#pragma unroll
                    for (int g = 0; g < kBN / 16; ++g)
                        // not 0: hidden scores stay -inf
                        c[g] = MOD == MOD_SOFTCAP ? k[g] * cap_in : fmaxf(k[g] * qk, 1e-37f);
                }
                if (take_turns && !turn_wait())
                    return;
                const int j0 = (first + kk * step) * kBN;
                if constexpr (MOD == MOD_SOFTCAP && F8) {
#pragma unroll
                    for (int g = 0; g < kBN / 16; ++g) {
                        softcap_scores<16>(*reinterpret_cast<float (*)[16]>(x + 16 * g), c[g], p.softcap_out);
                        c[g] = 1.f;
                    }
                } else if constexpr (MOD == MOD_SOFTCAP) {
                    softcap_scores<kBN>(x, p.softcap_in, p.softcap_out);
                }
                if (!(j0 >= full_lo && j0 + kBN <= full_hi))
                    apply_row_mask<kBN>(x, j0, row_lo, row_hi);
                uint32_t pk[kBN / 2];
                bool rescale;
                float alpha;
                if constexpr (F8) {
                    const uint32_t at = ptx::smem_u32(&sm.factors[t][(scount - 1) & 3]);
#pragma unroll
                    for (int i = 0; i < 8; i += 4)
                        ptx::load_shared_v4(at + 32 + 4 * i, log_v + i);
                    alpha = softmax_compute_p_scaled<kBN>(x, c, log_v, st, gap, pk, rescale);
                } else {
                    alpha = C::kOnes ? softmax_compute_p_exact_sum<kBN>(x, MOD == MOD_NONE ? p.qk_log2 : 1.f, st, false,
                                                                        pk, rescale)
                                     : softmax_compute_p<kBN>(x, MOD == MOD_NONE ? p.qk_log2 : 1.f, st, false, pk,
                                                              rescale);
                }
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
        float o_unit = 1.f;
        if constexpr (F8) {
            // the sum as one in [1, 2), m and O's unit to go with it: then O is no larger than
            // twice a value of V, whatever the scales are
            const float k = st.l == 0.f ? 0.f : static_cast<float>(static_cast<int>(__float_as_uint(st.l) >> 23) - 127);
            st.m_ref = (st.m_ref == kNegInf ? kNegInf : st.m_ref - gap + k);
            st.l *= ptx::ex2(-k);
            st.l_round = st.l; // P in f16 is within 2^-12 of it
            o_unit = ptx::ex2(gap - k) * ptx::ex2(-kPBias);
        }
        if (inf.pair) {
            if (active)
                write_slot<D, F8>(p, inf, t, r, tO, st, n_mine > 0, o_unit);
        } else {
            const uint32_t tX = cx.tmem + lanes + C::kColX;
            if (active) {
                const uint32_t ml[8] = {__float_as_uint(st.m_ref), __float_as_uint(st.l),
                                        __float_as_uint(st.l_round), __float_as_uint(o_unit), 0, 0, 0, 0};
                ptx::tmem_st8(tX + C::kStrideX * t, ml);
                ptx::tmem_wait_st();
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(sm.x_full[t]));
            if (!warp_wait(bar(sm.x_full[t ^ 1]), joins & 1, cx.wc, W_JOIN))
                return;
            ptx::tc_fence_after();
            if (active)
                write_joined<D, F8>(p, inf, t, r, tO, cx.tmem + lanes + C::kColO + C::kStrideO * (t ^ 1),
                                    tX + C::kStrideX * (t ^ 1), st, o_unit);
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(sm.x_free[t ^ 1])); // the other slot's O and sums have been read
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

// ------------------------------------------------------------------ kernel

// The kernel of the row blocks.
template <int MOD, int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkParams p)
{
    using C = ChunkCfg<D, F8>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    ChunkSmem<D, F8> *sm =
        reinterpret_cast<ChunkSmem<D, F8> *>(smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5;
    KernelCtx<D, F8> cx;
    cx.part = part_of(p);
    if (idle_second(p, 0, cx.part))
        return;

    for (uint32_t w = threadIdx.x; w < C::kOnesBytes / 4; w += kThreads)
        reinterpret_cast<uint32_t *>(sm->ones)[w] = 0x3F803F80u; // bf16 1.0 pairs
    ptx::fence_proxy_async_smem();
    if (threadIdx.x == 0) {
        ptx::prefetch_tensormap(&maps.q);
        ptx::prefetch_tensormap(&maps.k);
        ptx::prefetch_tensormap(&maps.v);
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar(sm->q_full[b]), 1);
            ptx::mbar_init(bar(sm->q_empty[b]), 1);
        }
        for (int b = 0; b < kInfo; ++b) {
            ptx::mbar_init(bar(sm->info_full[b]), 1);
            ptx::mbar_init(bar(sm->info_empty[b]), 11); // S, two P V and eight softmax warps
        }
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar(sm->kv_full[s]), F8 ? 1 + kScaleArrivals : 1);
            ptx::mbar_init(bar(sm->kv_empty[s]), F8 ? 3 : 2); // one arrival per P V warp, in 8 bits S's, too
        }
        for (int s = 0; s < (F8 ? C::kVStages : 0); ++s) {
            ptx::mbar_init(bar(sm->v_full[s]), 2); // one arrival per P V warp, here and below
            ptx::mbar_init(bar(sm->v_empty[s]), 2);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(bar(sm->s_full[t]), F8 ? 2 : 1); // the product, and its factors
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
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&sm->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();

    cx.sm = sm;
    cx.tmem = sm->tmem_base;
    cx.wc = wait_ctl(p, &sm->abort_flag);

    // each branch ends with its own copy of the teardown barrier, so no code
    // runs under both register limits
    if (warp >= 4) {
        ptx::setmaxnreg_inc<kRegsSoftmax>();
        tell_second(p, cx.part);
        softmax_role<MOD, D, F8>(cx, p, (warp >> 2) - 1);
        ptx::tc_fence_before();
        ptx::named_barrier_sync(1, kThreads);
    } else {
        ptx::setmaxnreg_dec<kRegsOther>();
        if (warp == 0)
            producer_role(cx, p, &maps.q, &maps.k, &maps.v);
        else if (warp == 1)
            s_role<MOD>(cx);
        else
            pv_role(cx, warp - 2);
        ptx::tc_fence_before();
        ptx::named_barrier_sync(1, kThreads);
        if (warp == 1) {
            ptx::tc_fence_after();
            ptx::tmem_dealloc(cx.tmem, 512);
        }
        ptx::wait_dependency(); // see chunk_plan.cuh
    }
}

// A launch that may start while the kernel before it in the stream runs (it
// waits for that one itself: ptx::wait_dependency).
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const Args &...args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Shared memory of a CTA, and the worst-case pad of its alignment.
template <class Smem>
constexpr size_t smem_bytes()
{
    static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory per CTA");
    return sizeof(Smem) + 1024;
}

template <int MOD, int D, bool F8>
cudaError_t configure(int device)
{
    static bool configured[64] = {}; // by device; benign race: the calls are idempotent
    if (configured[device])
        return cudaSuccess;
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, chunk_kernel<MOD, D, F8>);
    if (e != cudaSuccess)
        return e;
    // the setmaxnreg split assumes exactly kRegsLaunch registers at launch
    if (attr.numRegs != static_cast<int>(kRegsLaunch))
        return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(chunk_kernel<MOD, D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes<ChunkSmem<D, F8>>()));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chunk_few_kernel<MOD, D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem_bytes<FewSmem<D, F8>>()));
    configured[device] = e == cudaSuccess;
    return e;
}

template <int MOD, int D, bool F8>
cudaError_t launch_mod(const ChunkMaps &maps, ChunkParams &p, cudaStream_t stream)
{
    cudaError_t e = configure<MOD, D, F8>(p.device);
    if (e != cudaSuccess)
        return e;
    // one round of the planning kernel for the requests and their entries, as
    // long as its block allows, and a thread for each part
    int threads = 32;
    while (threads < kPlanThreads && (threads < p.batch || threads < p.max_entries))
        threads *= 2;
    const int block = std::min(std::max(threads, (2 * p.n_cta + 31) & ~31), kPlanThreads);
    // in 8 bits q is split beside it
    const int64_t rows = static_cast<int64_t>(p.T) * p.Hq, per_block = block / (D / 8) * kSplitRows;
    const int split = F8 ? static_cast<int>(std::min<int64_t>((rows + per_block - 1) / per_block, 4 * p.n_cta)) : 0;
    chunk_plan_kernel<D, F8><<<1 + split, block, 0, stream>>>(p, threads);
    e = cudaGetLastError();
    // groups of more than kFewRows heads have row blocks alone, and no more
    // tokens than few rows hold make no row block.  Where both may have work the
    // likelier one is first.
    const bool few = p.G <= kFewRows, blocks = !few || p.T > p.few_tq;
    const bool few_first = few && (!blocks || p.T <= static_cast<int64_t>(p.batch) * p.few_tq);
    if (!few || !blocks)
        p.seen_mark = 0;
    // the warm-up pays where the loads queue up: more keys than all rings hold
    p.warm = few_first && static_cast<double>(p.batch) * p.max_kv * p.Hk >
                              static_cast<double>(p.n_cta) * FewCfg<D, F8>::kStages * FewCfg<D, F8>::kBN;
    auto launch = [&](bool few_kernel) {
        const cudaError_t err = few_kernel
            ? launch_after(chunk_few_kernel<MOD, D, F8>, dim3(p.n_cta), kThreads, smem_bytes<FewSmem<D, F8>>(), stream, maps, p)
            : launch_after(chunk_kernel<MOD, D, F8>, dim3(p.n_cta), kThreads, smem_bytes<ChunkSmem<D, F8>>(), stream, maps, p);
        p.second = 1;
        p.warm = 0;
        return err;
    };
    if (e == cudaSuccess)
        e = launch(few_first);
    if (e == cudaSuccess && few && blocks)
        e = launch(!few_first);
    if (e != cudaSuccess)
        return e;
    return launch_after(chunk_join_kernel<D, F8>, dim3(p.n_cta, 2, kJoinSplit), kJoinThreads, 0, stream, p);
}

} // namespace
} // namespace fl
