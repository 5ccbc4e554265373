// fp8.cuh -- e4m3 on the way through the kernels of the 8-bit KV cache.
//
// A key's D codes stand for code * scale, scale by block of keys and KV head (fl_attn.h).
#pragma once

#include "chunk_plan.cuh"
#include "e4m3.cuh"
#include "softmax_tile.cuh"

namespace fl {
namespace {

// The scales of the last tiles, of K's and V's boxes of 16 keys.  The warp that loads
// K copies them along, and the barrier of the K tile covers them.  Who reads them has done so
// before the tile of 32 places on is loaded: loads are at most the rings and a few items
// ahead of the softmax (S of a tile waits for what its slot's last one was read for).
constexpr int kScaleRing = 32;
struct ScaleRing {
    float k[kScaleRing][16], v[kScaleRing][16];
};
constexpr int kScaleArrivals = 32; // on the tile's barrier: one per lane

// Copies the scales of the BOXES boxes from key0 on of request b; `page` is that of this
// lane's box of 2^page_box keys.  Boxes that no row sees and pages outside the cache get
// zeros.  A warp.
template <int BOXES>
__device__ __forceinline__ void copy_scales(const ChunkParams &p, ScaleRing &ring, uint32_t idx, uint32_t bar, int page,
                                            int page_box, int key0, int key_lo, int L, int kvh)
{
    const int lane = static_cast<int>(ptx::lane_id()), g = lane & 15, key = key0 + g * 16;
    const int pg = __shfl_sync(0xffffffffu, page, g * 16 >> page_box);
    const bool v = lane >= 16;
    const int at = p.page_shift < 0 ? key : key & ((1 << p.page_shift) - 1);
    const bool read = g < BOXES && key < L && key >= (key_lo & ~15) &&
                      static_cast<uint32_t>(pg) < static_cast<uint32_t>(p.n_pages);
    const float *from = v ? p.v_scale : p.k_scale;
    if (read)
        from += pg * (v ? p.vs_p : p.ks_p) + static_cast<int64_t>(at >> p.scale_shift) * (v ? p.vs_b : p.ks_b) + kvh;
    const uint32_t i = idx % kScaleRing;
    if (g < BOXES)
        ptx::copy_word(ptx::smem_u32(v ? &ring.v[i][g] : &ring.k[i][g]), from, read);
    ptx::copies_arrive(bar);
}

// Half `part` of the KEYS keys of a tile from codes (a key's D bytes after another's) to
// f16, which holds them exactly, in the layout of the 128-byte swizzle, halves of 64
// dimensions, by a warp.  Keys outside [dead_lo, dead_hi) become zero.  16 codes a lane and
// step: a 16-byte load and two 16-byte stores, 8 lanes of which meet in no bank.  Two steps
// of code: all seven in a row push the softmax's out of the instruction caches (2048
// softcapped tokens on 8192 keys 290 us, unrolled 328; without softcap 170 and 176).
template <int D, int KEYS>
__device__ __forceinline__ void convert_half(const uint8_t *raw, uint8_t *dst, int part, int dead_lo, int dead_hi)
{
    constexpr int kUnits = D / 16, kStepKeys = 32 / kUnits, kSteps = KEYS / 2 / kStepKeys;
    static_assert(kSteps * kStepKeys * 2 == KEYS, "whole steps");
    const int lane = static_cast<int>(ptx::lane_id()), u = lane % kUnits, key0 = part * (KEYS / 2) + lane / kUnits;
    const bool dead = dead_lo > 0 || dead_hi < KEYS;
    uint4 next = *reinterpret_cast<const uint4 *>(raw + key0 * D + u * 16);
#pragma unroll 2
    for (int i = 0; i < kSteps; ++i) {
        const int key = key0 + i * kStepKeys;
        uint4 w = next;
        if (i + 1 < kSteps)
            next = *reinterpret_cast<const uint4 *>(raw + (key + kStepKeys) * D + u * 16);
        if (dead && (key < dead_lo || key >= dead_hi))
            w = make_uint4(0, 0, 0, 0);
        uint4 out[2];
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t *o = reinterpret_cast<uint32_t *>(out);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            e4m3x4_to_f16x4(in[c], o[2 * c], o[2 * c + 1]);
        uint4 *row = reinterpret_cast<uint4 *>(dst + (u >> 2) * (KEYS * 128) + key * 128);
        const int at = (u & 3) * 2;
        row[at ^ (key & 7)] = out[0];
        row[(at + 1) ^ (key & 7)] = out[1];
    }
}

// The scales of a tile, as the softmax of row blocks takes them: of 16 keys each, K's and the logarithm
// of V's.  0 or NaN: a box that no row sees.
constexpr float kLeastLog = -110.f;
struct alignas(16) TileFactors {
    float k[8], log_v[8];
};

// By a warp; lane g < 8 has the scales of box g.
__device__ __forceinline__ void tile_factors(TileFactors &f, float k, float scale_v)
{
    const int lane = static_cast<int>(ptx::lane_id());
    if (lane < 8) {
        f.k[lane] = k > 0.f ? k : 0.f;
        f.log_v[lane] = fmaxf(ptx::lg2(scale_v), kLeastLog);
    }
}

// softmax_compute_p_exact_sum with a factor c of 16 scores each in place of one, and with V's
// scale in P, which multiplies V's codes: P = 2^(kPBias + z + log_v - m_ref) in f16, and the sum is
// relative to m = m_ref - gap, a reference of the scores alone.  Both references are the row's own:
// keys that it does not see have no say, however loud they are.  P stays below 2^(8 + kPBias), and
// holds 11 bits of a product of weight and scale down to 2^(-14 - kPBias) of the row's largest.
//
// The sum takes the same exponentials, times 2^(gap - kPBias - log_v) for 16 keys at a time.  Where
// log_v is 2^-kPSpread and more below the gap, P is below 2^(8 + kPBias - kPSpread) and 0 in f16; in its place
// stands that, and the sum's factor is as if log_v were that: so that neither goes out of
// range, whatever the scales are.
constexpr float kPBias = 6.f, kPSpread = 40.f;
template <int N>
__device__ __forceinline__ float softmax_compute_p_scaled(float (&x)[N], const float (&c)[N / 16],
                                                          const float (&log_v)[8], RowState &st, float &gap,
                                                          uint32_t (&pk)[N / 2], bool &rescale)
{
    float mp = kNegInf, mz = kNegInf;
#pragma unroll
    for (int g = 0; g < N / 16; ++g) {
        const float *s = x + 16 * g;
        float a = fmaxf(s[0], s[1]), b = fmaxf(s[2], s[3]);
#pragma unroll
        for (int e = 4; e < 16; e += 4) {
            a = ptx::max3(a, s[e], s[e + 1]);
            b = ptx::max3(b, s[e + 2], s[e + 3]);
        }
        const float z = fmaxf(a, b) * c[g]; // c > 0
        mz = fmaxf(mz, z);
        mp = fmaxf(mp, z + log_v[g]);
    }
    float alpha = 1.f;
    rescale = false;
    const float m = st.m_ref - gap;
    const bool need = mp > st.m_ref + kRescaleThreshold || mz > m + kRescaleThreshold;
    if (__any_sync(0xffffffffu, need)) {
        const float ref_new = fmaxf(st.m_ref, mp), m_new = fmaxf(m, mz);
        const bool none = ref_new == kNegInf;
        alpha = none ? 1.f : ptx::ex2(st.m_ref - ref_new);
        st.l *= none ? 1.f : ptx::ex2(m - m_new);
        st.m_ref = ref_new;
        gap = none ? 0.f : ref_new - m_new;
        rescale = true;
    }
    const float nmu = (st.m_ref == kNegInf) ? kPBias : kPBias - st.m_ref;
    const float least = gap - kPSpread, unit = gap - kPBias;
    float l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int g = 0; g < N / 16; ++g) {
        const float v = fmaxf(log_v[g], least), nm = nmu + v, f = ptx::ex2(unit - v);
        float le[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a0, a1;
            ptx::fma2(a0, a1, x[16 * g + 2 * e], x[16 * g + 2 * e + 1], c[g], c[g], nm, nm);
            const float p0 = ptx::ex2(a0), p1 = ptx::ex2(a1);
            pk[8 * g + e] = ptx::pack_f16(p0, p1);
            const int i = 2 * (e & 1);
            if (e < 2) {
                le[i] = p0;
                le[i + 1] = p1;
            } else {
                ptx::add2(le[i], le[i + 1], p0, p1);
            }
        }
        ptx::add2(le[0], le[1], le[2], le[3]);
        ptx::fma2(l0, l1, le[0], le[1], f, f, l0, l1);
    }
    st.l += l0 + l1;
    return alpha;
}

// Q as two e4m3 terms a row, relative to the row's scale: q = s (q1 + q2).  e4m3 has 4
// significant bits, what rounding to them leaves of bf16's 8 has 4 again, so the
// terms are exact for elements from 2^-10 of the row's largest on, and off by 2^-18 of
// it below.  A row with an element that is not finite becomes NaN there.  By the blocks
// of the planning kernel but the first; q8 [2][T][Hq][D], q_scale [T][Hq].
template <int D>
__device__ __forceinline__ void split_q(const ChunkParams &p)
{
    constexpr int kLanes = D / 8, kRows = kSplitRows; // lanes of a row, 8 elements each; rows a thread has in flight
    const int per = blockDim.x / kLanes, y = threadIdx.x / kLanes, u = threadIdx.x % kLanes;
    const int64_t rows = static_cast<int64_t>(p.T) * p.Hq;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x - 1) * per * kRows; r0 < rows;
         r0 += static_cast<int64_t>(gridDim.x - 1) * per * kRows) {
        uint4 in[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t r = r0 + k * per + y;
            in[k] = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const int64_t tok = rows >> 32 ? r / p.Hq : static_cast<uint32_t>(r) / static_cast<uint32_t>(p.Hq);
                in[k] = __ldg(reinterpret_cast<const uint4 *>(p.q + tok * p.q_st + (r - tok * p.Hq) * p.q_sh + u * 8));
            }
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t r = r0 + k * per + y;
            const uint32_t w[4] = {in[k].x, in[k].y, in[k].z, in[k].w};
            float x[8], m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                m = fmaxf(m, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
            }
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
                const uint32_t t = to_e4m3x2(lo, hi);
                const float2 v = from_e4m3x2(t);
                // an infinity saturates: its second term makes the sum NaN
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
    }
    ptx::fence_proxy_async_all(); // TMA reads it
}

} // namespace
} // namespace fl
