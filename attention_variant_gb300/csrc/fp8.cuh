// fp8.cuh -- e4m3 on the way through the kernels of the 8-bit KV cache.
//
// A key's D codes stand for code * scale, scale by block of keys and KV head
// (fl_attn.h).  e4m3 has 4 significant bits, bf16 has 8: where the scale is a power of
// two, code * scale is a bf16 number, and the conversion is exact.
//
// A byte s eeee mmm shifted to where bf16 has its sign, the low bits of its exponent
// and the high ones of its mantissa stands for 2^-120 times its value, subnormals
// too, so one packed multiplication by 2^120 scale finishes two of them.  (The
// NaN codes come out as +-480.)
#pragma once

#include "chunk_plan.cuh"
#include "e4m3.cuh"

namespace fl {
namespace {

constexpr int kConvertThreads = 128; // four warps

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The multipliers of a block of codes: value = bits * first * second.  Their product,
// 2^120 scale, may exceed bf16's range; scales up to 2^7 need the first alone.
struct Fp8Scale {
    uint32_t first, second;
    bool one;
};
__device__ __forceinline__ Fp8Scale fp8_scale(float scale)
{
    Fp8Scale f;
    f.one = !(scale > 64.f);
    const float a = f.one ? scale * 0x1p120f : 0x1p126f, b = f.one ? 1.f : scale * 0x1p-6f;
    f.first = ptx::pack_bf16(a, a);
    f.second = ptx::pack_bf16(b, b);
    return f;
}

// Four codes -> two words of two bf16.
__device__ __forceinline__ uint2 fp8_to_bf16(uint32_t w, const Fp8Scale &f)
{
    uint32_t out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t t = __byte_perm(w, 0, i ? 0x3424 : 0x1404); // each code in the high byte of its half
        const uint32_t bits = ((t & 0x7f007f00u) >> 4) | (t & 0x80008000u);
        out[i] = mul_bf16x2(bits, f.first);
    }
    if (!f.one) {
        out[0] = mul_bf16x2(out[0], f.second);
        out[1] = mul_bf16x2(out[1], f.second);
    }
    return make_uint2(out[0], out[1]);
}

// The scale of a key of request b.  Keys that no row sees and pages outside the
// cache have none.
__device__ __forceinline__ float box_scale(const ChunkParams &p, const float *scale, int64_t s_page, int64_t s_block,
                                           int b, int key, int key_lo, int L, int kvh)
{
    if (key >= L || key < key_lo)
        return 0.f;
    int page = b, at = key;
    if (p.page_shift >= 0) {
        page = __ldg(p.block_table + static_cast<int64_t>(b) * p.bt_stride + (key >> p.page_shift));
        at = key & ((1 << p.page_shift) - 1);
    }
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.n_pages))
        return 0.f;
    return __ldg(scale + page * s_page + static_cast<int64_t>(at >> p.scale_shift) * s_block + kvh);
}

// The scales of a tile's boxes of 16 keys in the lanes of a warp.  (A box that holds
// some key that a row sees has that key's.)
__device__ __forceinline__ float tile_scales(const ChunkParams &p, const float *scale, int64_t s_page, int64_t s_block,
                                             int b, int key0, int key_lo, int L, int kvh)
{
    const int lane = static_cast<int>(ptx::lane_id());
    return lane < 8 ? box_scale(p, scale, s_page, s_block, b, key0 + lane * 16, key_lo & ~15, L, kvh) : 0.f;
}

// A tile of KEYS keys from codes (a key's D bytes after another's) to bf16 in the layout
// of the 128-byte swizzle, halves of 64 dimensions, by four warps.  Keys outside
// [dead_lo, dead_hi) become zero.  16 codes a thread and step: a 16-byte load (all of
// them first) and two 16-byte stores, 8 threads of which meet in no bank.
template <int D, int KEYS>
__device__ __forceinline__ void convert_tile(const uint8_t *raw, uint8_t *dst, float scales, int dead_lo, int dead_hi)
{
    constexpr int kUnits = D / 16, kSteps = (KEYS * kUnits + kConvertThreads - 1) / kConvertThreads;
    constexpr bool kRagged = KEYS * kUnits % kConvertThreads != 0; // the last step is some warps' alone
    const int tid = threadIdx.x & (kConvertThreads - 1), u = tid % kUnits;
    uint4 w[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if (!kRagged || i + 1 < kSteps || tid + i * kConvertThreads < KEYS * kUnits)
            w[i] = *reinterpret_cast<const uint4 *>(raw + (tid + i * kConvertThreads) * 16);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int key = tid / kUnits + i * (kConvertThreads / kUnits);
        const Fp8Scale f = fp8_scale(__shfl_sync(0xffffffffu, scales, (key >> 4) & 7));
        if (kRagged && i + 1 == kSteps && tid + i * kConvertThreads >= KEYS * kUnits)
            break;
        uint4 out[2];
        const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t *o = reinterpret_cast<uint32_t *>(out);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint2 y = fp8_to_bf16(in[c], f);
            o[2 * c] = y.x;
            o[2 * c + 1] = y.y;
        }
        if (key < dead_lo || key >= dead_hi)
            out[0] = out[1] = make_uint4(0, 0, 0, 0);
        uint4 *row = reinterpret_cast<uint4 *>(dst + (u >> 2) * (KEYS * 128) + key * 128);
        const int at = (u & 3) * 2;
        row[at ^ (key & 7)] = out[0];
        row[(at + 1) ^ (key & 7)] = out[1];
    }
}

// Q as two e4m3 terms a row, relative to the row's scale: q = s (q1 + q2).  e4m3 has 4
// significant bits, what rounding to them leaves of bf16's 8 has 4 again, so the
// terms are exact for elements from 2^-10 of the row's largest on, and off by 2^-18 of
// it below.  A row with an element that is not finite becomes NaN there.  By the blocks
// of the planning kernel but the first; q8 [2][T][Hq][D], q_scale [T][Hq].
template <int D>
__device__ __forceinline__ void split_q(const ChunkParams &p)
{
    constexpr int kLanes = D / 8; // of a row, 8 elements each
    const int per = blockDim.x / kLanes, y = threadIdx.x / kLanes, u = threadIdx.x % kLanes;
    const int64_t rows = static_cast<int64_t>(p.T) * p.Hq;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x - 1) * per; r0 < rows; r0 += static_cast<int64_t>(gridDim.x - 1) * per) {
        const int64_t r = r0 + y, tok = r / p.Hq;
        float x[8];
        if (r < rows) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p.q + tok * p.q_st + (r - tok * p.Hq) * p.q_sh + u * 8));
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(in[i] << 16);
                x[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = 0.f;
        }
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = fmaxf(m, fabsf(x[i]));
#pragma unroll
        for (int d = kLanes / 2; d; d >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (r >= rows)
            continue;
        const uint32_t s = m < -kNegInf ? scale_bits(__float_as_uint(m)) : 0x3f800000u;
        const float inv = __uint_as_float((254u << 23) - s); // 1 / s, s a power of two
        uint32_t a[2] = {0, 0}, b[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = x[2 * i] * inv, hi = x[2 * i + 1] * inv;
            // an infinity saturates; its difference from that makes the second term's sum NaN
            const uint32_t t = to_e4m3x2(lo, hi);
            const float2 v = from_e4m3x2(t);
            const float l2 = fabsf(lo) < -kNegInf ? lo - v.x : __uint_as_float(0x7fffffffu);
            const float h2 = fabsf(hi) < -kNegInf ? hi - v.y : __uint_as_float(0x7fffffffu);
            a[i >> 1] |= t << (16 * (i & 1));
            b[i >> 1] |= to_e4m3x2(l2, h2) << (16 * (i & 1));
        }
        uint8_t *dst = p.q8 + r * D + u * 8;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(a[0], a[1]);
        *reinterpret_cast<uint2 *>(dst + rows * D) = make_uint2(b[0], b[1]);
        if (u == 0)
            p.q_scale[r] = __uint_as_float(s);
    }
    ptx::fence_proxy_async_all(); // TMA reads it
}

} // namespace
} // namespace fl
