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

// A scale of the cache: of the 16 keys from `key` on of request b.  Keys past the
// last and pages outside the cache have none.
__device__ __forceinline__ float box_scale(const ChunkParams &p, const float *scale, int64_t s_page, int64_t s_block,
                                           int b, int key, int L, int kvh)
{
    if (key >= L)
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

// The scales of tile j in the lanes of a warp: those of K's boxes of 16 keys in
// lanes 0 .. 7, of V's in 8 .. 15.
__device__ __forceinline__ float tile_scales(const ChunkParams &p, int b, int key0, int L, int kvh)
{
    const int lane = static_cast<int>(ptx::lane_id()), key = key0 + (lane & 7) * 16;
    if (lane >= 16)
        return 0.f;
    return lane < 8 ? box_scale(p, p.k_scale, p.ks_p, p.ks_b, b, key, L, kvh)
                    : box_scale(p, p.v_scale, p.vs_p, p.vs_b, b, key, L, kvh);
}

// A tile of KEYS keys from codes (a key's D bytes after another's) to bf16 in the layout
// of the 128-byte swizzle, halves of 64 dimensions, by four warps.  Keys outside
// [dead_lo, dead_hi) become zero.  `scales`: tile_scales, from lane `from` on.
// 16 codes a thread and step: a 16-byte load and two 16-byte stores, 8 threads of
// which meet in no bank.
template <int D, int KEYS>
__device__ __forceinline__ void convert_tile(const uint8_t *raw, uint8_t *dst, float scales, int from, int dead_lo,
                                             int dead_hi)
{
    constexpr int kUnits = D / 16; // of a key
    const int tid = threadIdx.x & (kConvertThreads - 1);
#pragma unroll
    for (int c0 = 0; c0 < KEYS * kUnits; c0 += kConvertThreads) {
        const int c = c0 + tid, key = c / kUnits, u = c % kUnits;
        if (KEYS * kUnits % kConvertThreads && c >= KEYS * kUnits) // whole warps
            break;
        const Fp8Scale f = fp8_scale(__shfl_sync(0xffffffffu, scales, from + (key >> 4)));
        const uint4 w = *reinterpret_cast<const uint4 *>(raw + c * 16);
        uint4 out[2];
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t *o = reinterpret_cast<uint32_t *>(out);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 y = fp8_to_bf16(in[i], f);
            o[2 * i] = y.x;
            o[2 * i + 1] = y.y;
        }
        if (key < dead_lo || key >= dead_hi)
            out[0] = out[1] = make_uint4(0, 0, 0, 0);
        uint4 *row = reinterpret_cast<uint4 *>(dst + (u >> 2) * (KEYS * 128) + key * 128);
        const int at = (u & 3) * 2;
        row[at ^ (key & 7)] = out[0];
        row[(at + 1) ^ (key & 7)] = out[1];
    }
}

} // namespace
} // namespace fl
