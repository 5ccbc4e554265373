// rope.cuh -- the rotation of rope.cu (see there), shared with the append to a
// cache in 8 bits.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "common.cuh"
#include "launch.h"

namespace fl {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRows = 8;         // (token, head) rows per thread, where there are enough
constexpr int kMaxAngles = 1024; // tokens of a tile times pairs
constexpr int kMaxTile = 64;

template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float &d, float x) { d = x; }
__device__ __forceinline__ void narrow(__nv_bfloat16 &d, float x) { d = __float2bfloat16(x); }

// cos and sin of `turn` / 2^64 turns.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t turn)
{
    const uint32_t hi = static_cast<uint32_t>(turn >> 32);
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(hi - (quarter << 30)); // [-2^29, 2^29)
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    switch (quarter & 3u) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
    }
}

// Where the angle of a token's pair i lies: two angles (16 bytes) of each unit
// of V pairs, then the next two of each, so that the threads of neighbouring
// units read neighbouring words (unit after unit, 8 threads met in two groups
// of banks: 29.5 us for the append of 11,810 tokens of 16 + 2 + 2 heads of 128,
// 27.8 this way).
template <int V>
__device__ __forceinline__ int angle_at(int i, int units)
{
    if constexpr (V <= 2)
        return i;
    const int u = i / V, e = i % V;
    return ((e / 2) * units + u) * 2 + e % 2;
}

// Rotates the V pairs of (a, b) by the angles of their unit, cs[angle_at]:
// pair e is (a, b)[e], or, where INTER, neighbours of the 2 V elements a, b.
template <class T, int V, bool INTER>
__device__ __forceinline__ void rotate_pairs(Vec<T, V> &a, Vec<T, V> &b, const float2 *cs, int units)
{
    if constexpr (sizeof(T) == 2 && V >= 2) {
        // bf16 two at a time: a word holds pairs e, e + 1 of one half, or both
        // elements of a pair; widening is a shift or a mask, narrowing one cvt
        uint32_t *wa = reinterpret_cast<uint32_t *>(&a), *wb = reinterpret_cast<uint32_t *>(&b);
        auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
        auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            // cos, sin of pairs e, e + 1
            const float4 f = *reinterpret_cast<const float4 *>(cs + e * units);
            uint32_t &w0 = INTER ? (e < V / 2 ? wa[e % (V / 2)] : wb[e % (V / 2)]) : wa[e / 2];
            uint32_t &w1 = INTER ? (e + 1 < V / 2 ? wa[(e + 1) % (V / 2)] : wb[(e + 1) % (V / 2)]) : wb[e / 2];
            const float a0 = lo(w0), b0 = INTER ? hi(w0) : lo(w1);
            const float a1 = INTER ? lo(w1) : hi(w0), b1 = hi(w1);
            const float ya0 = a0 * f.x - b0 * f.y, yb0 = a0 * f.y + b0 * f.x;
            const float ya1 = a1 * f.z - b1 * f.w, yb1 = a1 * f.w + b1 * f.z;
            w0 = INTER ? ptx::pack_bf16(ya0, yb0) : ptx::pack_bf16(ya0, ya1);
            w1 = INTER ? ptx::pack_bf16(ya1, yb1) : ptx::pack_bf16(yb0, yb1);
        }
    } else {
        alignas(16) float2 f[V];
        if constexpr (V == 1)
            f[0] = cs[0];
        else
#pragma unroll
            for (int e = 0; e < V; e += 2)
                *reinterpret_cast<float4 *>(f + e) = *reinterpret_cast<const float4 *>(cs + e * units);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            T &ra = INTER ? (2 * e < V ? a.e[(2 * e) % V] : b.e[(2 * e) % V]) : a.e[e];
            T &rb = INTER ? (2 * e + 1 < V ? a.e[(2 * e + 1) % V] : b.e[(2 * e + 1) % V]) : b.e[e];
            const float xa = widen(ra), xb = widen(rb);
            narrow(ra, xa * f[e].x - xb * f[e].y);
            narrow(rb, xa * f[e].y + xb * f[e].x);
        }
    }
}

// A block's share of one tensor.  s_cs: kMaxAngles; s_src, s_dst: kMaxTile, rows of
// the tile's tokens (s_dst < 0: skipped).
template <class T, int V, bool INTER>
__device__ __forceinline__ void rope_tile(const RopeParams &p, const RopeStream &st, float2 *s_cs, int64_t *s_src,
                                          int64_t *s_dst)
{
    const int rot_units = p.pairs / V;
    const int tid = threadIdx.x, t0 = blockIdx.x * st.tile, n_tok = min(st.tile, p.tokens - t0);
    if (n_tok <= 0)
        return; // the grid is as wide as the tensor with the smallest tiles needs

    if (tid < n_tok) {
        const int t = t0 + tid, b = fast_div(t, p.div_seq), s = t - b * p.div_seq.d;
        int64_t dst = b * st.d_b + s * st.d_s;
        if (p.slots) {
            const int64_t slot = __ldg(p.slots + t);
            if (slot < 0 || slot >= p.n_slots) {
                dst = -1;
            } else if (st.to_cache) {
                const int64_t page = slot / p.page_rows;
                dst = page * st.d_b + (slot - page * p.page_rows) * st.d_s;
            }
        }
        s_src[tid] = b * st.s_b + s * st.s_s;
        s_dst[tid] = dst;
    }
    if (st.rotate) {
        // frequencies are constants, which the lanes of a warp fetch one after another: a
        // thread keeps its own, the same one throughout where the pairs divide the threads
        // (append of 11,810 tokens of 16 + 2 + 2 heads of 128: 28.0 -> 24.5 us)
        int turn_i = -1;
        uint64_t turn = 0;
        for (int e = tid; e < n_tok * p.pairs; e += kRopeThreads) {
            const int tl = fast_div(e, p.div_pairs), i = e - tl * p.pairs;
            const int t = t0 + tl, b = fast_div(t, p.div_seq), s = t - b * p.div_seq.d;
            const int64_t pos = p.offset + (p.positions ? __ldg(p.positions + b * p.positions_stride + s) : s);
            if (i != turn_i) {
                turn_i = i;
                turn = p.turns[i];
            }
            float2 cs = turn_cos_sin(static_cast<uint64_t>(pos) * turn);
            cs.x *= p.magnitude;
            cs.y *= p.backward ? -p.magnitude : p.magnitude;
            s_cs[tl * p.pairs + angle_at<V>(i, rot_units)] = cs;
        }
    }
    __syncthreads();

    // unit ux of a head: the vectors a (at element `at`) and b (b_at further) of
    // V rotated pairs, or one vector of the copied rest (b_at 0)
    const int y = fast_div(tid, p.div_ux), x = tid - y * p.div_ux.d;
    if (y >= p.uy)
        return;
    const int rows = n_tok * st.heads;
    for (int ux = x; ux < p.units; ux += p.div_ux.d) {
        const bool pair = ux < rot_units;
        const int at = !pair ? p.rot + (ux - rot_units) * V : INTER ? ux * 2 * V : ux * V;
        const int b_at = INTER ? V : p.pairs;
        const T *src = static_cast<const T *>(st.src) + at;
        T *dst = static_cast<T *>(st.dst) + at;
        for (int r = y; r < rows; r += p.uy) {
            const int tok = fast_div(r, st.div_heads), h = r - tok * st.heads;
            if (s_dst[tok] < 0)
                continue;
            const T *from = src + s_src[tok] + h * st.s_h;
            T *to = dst + s_dst[tok] + h * st.d_h;
            Vec<T, V> a = *reinterpret_cast<const Vec<T, V> *>(from), b;
            if (pair) {
                b = *reinterpret_cast<const Vec<T, V> *>(from + b_at);
                if (st.rotate)
                    rotate_pairs<T, V, INTER>(a, b, s_cs + tok * p.pairs + ux * (V == 1 ? 1 : 2), rot_units);
                *reinterpret_cast<Vec<T, V> *>(to + b_at) = b;
            }
            *reinterpret_cast<Vec<T, V> *>(to) = a;
        }
    }
}

// Units, and tokens per block of each tensor; the blocks that takes (0: nothing to do).
inline int rope_shape(RopeParams &p, int vec, int sm_count)
{
    p.units = p.pairs / vec + p.pass / vec;
    if (p.units == 0 || p.tokens == 0)
        return 0;
    const int ux = p.units < kRopeThreads ? p.units : kRopeThreads;
    p.div_ux = make_fastdiv(ux);
    p.uy = kRopeThreads / ux;
    // tokens per block: as many as give each thread its kRows rows, as long as
    // the tensor still fills the GPU's block slots about twice
    int blocks = 0;
    for (int i = 0; i < p.n_streams; ++i) {
        RopeStream &st = p.st[i];
        int tile = 1;
        while (tile < kMaxTile && 2 * int64_t(tile) * st.heads <= kRows * p.uy && 2 * tile * p.pairs <= kMaxAngles &&
               p.tokens / (2 * tile) >= 4 * sm_count)
            tile *= 2;
        st.tile = tile;
        const int n = (p.tokens + tile - 1) / tile;
        blocks = n > blocks ? n : blocks;
    }
    return blocks;
}

} // namespace
} // namespace fl
