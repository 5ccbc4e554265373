// rope.cu -- rotary positions of q and k, and the same on the way into a
// paged KV cache (the append of new keys and values).
//
//   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_a sin t + x_b cos t),  t = pos f_i
//
// The angle: f_i / 2 pi is held as a 64-bit fraction of a turn, so pos times
// it, in 64-bit integers, is the angle modulo a turn with no reduction and no
// error that grows with the position (a 32-bit float angle is off by 0.06 rad
// at position 10^6).  The nearest quarter turn is taken off in integers too;
// the remainder, in [-1/8, 1/8] turn, goes to sincospif.
//
// Bound by HBM: every element is read and written once.  A block takes `tile`
// tokens, puts their sines and cosines in shared memory (one sincos for all
// heads of a token) and streams all heads of all tensors through, a thread
// moving the two vectors of up to 16 bytes that hold its pairs' halves.  The
// vectors are loaded before the sines are ready, so both latencies overlap.
#include <cuda_bf16.h>
#include <cstdint>

#include "common.cuh"
#include "launch.h"

namespace fl {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;      // units in flight per thread
constexpr int kMaxAngles = 1024; // tokens of a tile times pairs

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

// A unit: the two vectors that hold V rotated pairs (a, b), or one vector of
// V elements that are copied (b unused).
template <class T, int V>
struct Unit {
    Vec<T, V> a, b;
    T *dst;      // of a; null: nothing to store
    int b_at;    // b's distance from a; 0: a copied unit
    int angle;   // first pair's place in the table of the tile; < 0: not rotated
};

template <class T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ float2 s_cs[kMaxAngles];
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.tile;
    const int n_tok = min(p.tile, p.tokens - t0);
    const int total = n_tok * p.heads * p.units;
    const int rot_units = p.pairs / V;

    auto load = [&](int u, Unit<T, V> &w) {
        w.dst = nullptr;
        if (u >= total)
            return;
        const int tl = fast_div(u, p.div_head_units);
        const int in_tok = u - tl * p.div_head_units.d;
        int h = fast_div(in_tok, p.div_units);
        const int un = in_tok - h * p.units;
        int si = 0;
        while (si + 1 < p.n_streams && h >= p.st[si].heads)
            h -= p.st[si++].heads;
        const RopeStream &st = p.st[si];
        const int t = t0 + tl;
        const int b = fast_div(t, p.div_seq), s = t - b * p.div_seq.d;
        int64_t d_row;
        if (st.to_cache) {
            const int64_t slot = __ldg(p.slots + t);
            if (slot < 0 || slot >= p.n_slots)
                return;
            const int64_t page = slot / p.div_tile_page.d;
            d_row = page * st.d_b + (slot - page * p.div_tile_page.d) * st.d_s;
        } else {
            if (p.slots) {
                const int64_t slot = __ldg(p.slots + t);
                if (slot < 0 || slot >= p.n_slots)
                    return;
            }
            d_row = b * st.d_b + s * st.d_s;
        }
        int at; // element of the head where a starts
        w.angle = -1;
        if (un < rot_units) {
            at = INTER ? un * 2 * V : un * V;
            w.b_at = INTER ? V : p.pairs;
            if (st.rotate)
                w.angle = tl * p.pairs + un * V;
        } else {
            at = p.rot + (un - rot_units) * V;
            w.b_at = 0;
        }
        const T *src = static_cast<const T *>(st.src) + b * st.s_b + s * st.s_s + h * st.s_h + at;
        w.a = *reinterpret_cast<const Vec<T, V> *>(src);
        if (w.b_at)
            w.b = *reinterpret_cast<const Vec<T, V> *>(src + w.b_at);
        w.dst = static_cast<T *>(st.dst) + d_row + h * st.d_h + at;
    };
    auto store = [&](Unit<T, V> &w) {
        if (!w.dst)
            return;
        if (w.angle >= 0) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 cs = s_cs[w.angle + e];
                T &ra = INTER ? (2 * e < V ? w.a.e[(2 * e) % V] : w.b.e[(2 * e) % V]) : w.a.e[e];
                T &rb = INTER ? (2 * e + 1 < V ? w.a.e[(2 * e + 1) % V] : w.b.e[(2 * e + 1) % V]) : w.b.e[e];
                const float xa = widen(ra), xb = widen(rb);
                narrow(ra, xa * cs.x - xb * cs.y);
                narrow(rb, xa * cs.y + xb * cs.x);
            }
        }
        *reinterpret_cast<Vec<T, V> *>(w.dst) = w.a;
        if (w.b_at)
            *reinterpret_cast<Vec<T, V> *>(w.dst + w.b_at) = w.b;
    };

    Unit<T, V> w[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
        load(tid + k * kThreads, w[k]);
    for (int e = tid; e < n_tok * p.pairs; e += kThreads) {
        const int tl = e / p.pairs, i = e - tl * p.pairs;
        const int t = t0 + tl;
        const int b = fast_div(t, p.div_seq), s = t - b * p.div_seq.d;
        const int64_t pos = p.offset + (p.positions ? __ldg(p.positions + b * p.positions_stride + s) : s);
        float2 cs = turn_cos_sin(static_cast<uint64_t>(pos) * p.turns[i]);
        cs.x *= p.magnitude;
        cs.y *= p.backward ? -p.magnitude : p.magnitude;
        s_cs[e] = cs;
    }
    __syncthreads();
    for (int u = tid;;) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            store(w[k]);
        u += kUnroll * kThreads;
        if (u >= total)
            break;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            load(u + k * kThreads, w[k]);
    }
}

template <class T, int V>
cudaError_t launch_vec(RopeParams &p, bool interleaved, int sm_count, cudaStream_t stream)
{
    p.units = p.pairs / V + p.pass / V;
    const int64_t head_units = int64_t(p.heads) * p.units;
    if (head_units == 0 || p.tokens == 0)
        return cudaSuccess;
    // tokens per block: as many as fill a block's first kUnroll rounds and its
    // table, as long as two blocks a SM remain
    int tile = 1;
    while (tile < 64 && 2 * tile * head_units <= kThreads * kUnroll && 2 * tile * p.pairs <= kMaxAngles &&
           p.tokens / (2 * tile) >= 2 * sm_count)
        tile *= 2;
    p.tile = tile;
    p.div_units = make_fastdiv(p.units);
    p.div_head_units = make_fastdiv(static_cast<int32_t>(head_units));
    const int grid = (p.tokens + tile - 1) / tile;
    if (interleaved)
        rope_kernel<T, V, true><<<grid, kThreads, 0, stream>>>(p);
    else
        rope_kernel<T, V, false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_rope(const RopeParams &params, bool fp32, bool interleaved, int vec, int sm_count,
                        cudaStream_t stream)
{
    RopeParams p = params;
    if (fp32) {
        if (vec >= 4)
            return launch_vec<float, 4>(p, interleaved, sm_count, stream);
        if (vec == 2)
            return launch_vec<float, 2>(p, interleaved, sm_count, stream);
        return launch_vec<float, 1>(p, interleaved, sm_count, stream);
    }
    if (vec >= 8)
        return launch_vec<__nv_bfloat16, 8>(p, interleaved, sm_count, stream);
    if (vec == 4)
        return launch_vec<__nv_bfloat16, 4>(p, interleaved, sm_count, stream);
    if (vec == 2)
        return launch_vec<__nv_bfloat16, 2>(p, interleaved, sm_count, stream);
    return launch_vec<__nv_bfloat16, 1>(p, interleaved, sm_count, stream);
}

} // namespace fl
