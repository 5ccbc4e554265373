// kv_fp8.cu -- new keys and values into a paged cache of e4m3 codes, rotated on
// the way, and tokens of such a cache read back.
//
//   code = rn(x / s),  s the scale of the row's block of keys and head
//
// s is the smallest power of two that 448 s holds every finite |x| of the block,
// at least 2^-100: then x / s is exact, and a scale that grows leaves codes c -> rn(c
// s_old / s), which rounds subnormals alone.  So the codes of a block hardly depend on how
// its tokens were split over calls, and its scale not at all.
//
// The tokens of a block that a call brings are neighbours (fl_kv_plan lists them
// so): a run.  A thread block takes the runs that begin among its tokens one after
// another, for a group of heads: each thread keeps its 16 elements of up to four
// (token, head) rows in registers, rotated, from the maximum (over the lanes of a row, then in
// shared memory) to the codes.  Runs too long for that are read and rotated twice, the
// second time out of L2.  Bound by HBM; for single tokens by the launch and one chain of
// loads.
#include <cuda_bf16.h>
#include <cstdint>

#include "e4m3.cuh"
#include "rope.cuh"

namespace fl {
namespace {

constexpr int kRowsKept = 4;      // (token, head) rows a thread keeps
constexpr int kRunAngles = 4096;  // tokens of a chunk times pairs
constexpr int kRunHeads = 16;     // heads of a group, at most

struct RunShared {
    float2 cs[kRunAngles];
    int row[256];              // rows in the block of the chunk's tokens
    uint32_t size[kRunHeads];  // largest |x| of each head, as bits
    uint32_t old[kRunHeads];   // its scale before
    int n;                     // tokens of the chunk
    int fresh;                 // the block's first row is among the run's
};

// Where a thread's unit k of 2 V elements lies: vector a at the first place, b
// `b_at` further (V elements each).
template <int V, bool INTER, bool ROT>
__device__ __forceinline__ int unit_at(int u, int rot_units, int rot, int pairs, int &b_at)
{
    b_at = V;
    if (!ROT || u >= rot_units)
        return rot + (u - rot_units) * 2 * V;
    if (INTER)
        return u * 2 * V;
    b_at = pairs;
    return u * V;
}

// The runs that begin among the block's tokens, for heads h0 .. h0 + group - 1.
template <int V, bool INTER, bool ROT>
__device__ __forceinline__ void append_runs(const Fp8AppendParams &f, const Fp8Stream &st, int h0, RunShared &sm)
{
    constexpr int kUnits = 8 / V; // of a thread's 16 elements
    const RopeParams &p = f.rope;
    const int tid = threadIdx.x, lane = tid & 31;
    const int lpr = 1 << f.lane_shift, piece = tid & (lpr - 1), y = tid >> f.lane_shift, rp = kRopeThreads >> f.lane_shift;
    const int rot = ROT ? p.rot : 0, pairs = ROT ? p.pairs : 0, rot_units = pairs / V;
    const int t0 = blockIdx.x * f.tile, sb = 1 << f.block_shift;
    auto block_of = [&](int t) { // -1: skipped
        const int64_t slot = t >= 0 && t < p.tokens ? __ldg(p.slots + t) : -1;
        return slot < 0 || slot >= p.n_slots ? int64_t(-1) : slot >> f.block_shift;
    };
    // every warp finds the runs for itself
    uint32_t runs;
    {
        const int64_t mine = lane < f.tile ? block_of(t0 + lane) : -1;
        const int64_t before = lane < f.tile ? block_of(t0 + lane - 1) : -1;
        runs = __ballot_sync(0xffffffffu, mine >= 0 && mine != before);
    }
    for (; runs; runs &= runs - 1) {
        const int start = t0 + __ffs(runs) - 1;
        const int64_t blk = block_of(start);
        const int64_t page = (blk << f.block_shift) / p.page_rows;
        const int first_row = static_cast<int>((blk << f.block_shift) - page * p.page_rows);
        uint8_t *const cache = st.cache + page * st.d_p + first_row * st.d_r + h0 * st.d_h;
        float *const scale = st.scale + page * st.s_p + (first_row >> f.block_shift) * st.s_b + h0;
        float x[kRowsKept][16];

        // the chunk's tokens: their number, and rows in the block
        auto find = [&](int c0) {
            __syncthreads(); // the last chunk's have been read
            if (tid == 0)
                sm.n = f.chunk;
            __syncthreads();
            if (tid < f.chunk) {
                if (block_of(c0 + tid) != blk)
                    atomicMin(&sm.n, tid);
                else
                    sm.row[tid] = static_cast<int>(__ldg(p.slots + c0 + tid) & (sb - 1));
            }
            __syncthreads();
            const int n = sm.n;
            if (tid < n && sm.row[tid] == 0)
                sm.fresh = 1;
            if constexpr (ROT) {
                for (int e = tid; e < n * pairs; e += kRopeThreads) {
                    const int tl = fast_div(e, p.div_pairs), i = e - tl * pairs;
                    float2 cs = turn_cos_sin(static_cast<uint64_t>(p.offset + __ldg(p.positions + c0 + tl)) * p.turns[i]);
                    cs.x *= p.magnitude;
                    cs.y *= p.magnitude;
                    sm.cs[tl * pairs + angle_at<V>(i, rot_units)] = cs;
                }
                __syncthreads();
            }
            return n;
        };
        // this thread's elements of its rows, rotated; what is infinite is not a number
        auto load = [&](int c0, int n, bool measure) {
#pragma unroll
            for (int i = 0; i < kRowsKept; ++i) {
                const int r = y + i * rp, tok = fast_div(r, f.div_group), h = r - tok * f.div_group.d;
                const bool live = tok < n;
                if (live) {
                    const __nv_bfloat16 *src = st.src + static_cast<int64_t>(c0 + tok) * st.s_s + (h0 + h) * st.s_h;
#pragma unroll
                    for (int k = 0; k < kUnits; ++k) {
                        const int u = piece * kUnits + k;
                        int b_at;
                        const int at = unit_at<V, INTER, ROT>(u, rot_units, rot, pairs, b_at);
                        const auto a = *reinterpret_cast<const Vec<__nv_bfloat16, V> *>(src + at);
                        const auto b = *reinterpret_cast<const Vec<__nv_bfloat16, V> *>(src + at + b_at);
                        float *w = x[i] + k * 2 * V; // V elements of a, V of b
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            w[e] = __bfloat162float(a.e[e]);
                            w[V + e] = __bfloat162float(b.e[e]);
                        }
                        if (ROT && u < rot_units) {
                            const float2 *cs = sm.cs + tok * pairs + u * (V == 1 ? 1 : 2);
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                const float2 t = V <= 2 ? cs[e] : cs[(e / 2) * rot_units * 2 + e % 2];
                                float &ra = INTER ? w[2 * e] : w[e], &rb = INTER ? w[2 * e + 1] : w[V + e];
                                const float xa = ra, xb = rb;
                                ra = xa * t.x - xb * t.y;
                                rb = xa * t.y + xb * t.x;
                            }
                        }
                    }
                }
                float m = 0.f;
                if (live) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        m = fmaxf(m, fabsf(x[i][e]));
                    if (m == -kNegInf) {
                        m = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (fabsf(x[i][e]) == -kNegInf)
                                x[i][e] = __uint_as_float(0x7fffffffu);
                            else
                                m = fmaxf(m, fabsf(x[i][e]));
                        }
                    }
                }
                if (!measure)
                    continue;
                uint32_t top = __float_as_uint(m);
                for (int d = lpr / 2; d; d >>= 1)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                if (live && piece == 0 && top)
                    atomicMax(&sm.size[h], top);
            }
        };
        auto store = [&](int n) {
#pragma unroll
            for (int i = 0; i < kRowsKept; ++i) {
                const int r = y + i * rp, tok = fast_div(r, f.div_group), h = r - tok * f.div_group.d;
                if (tok >= n)
                    continue;
                const float s = __uint_as_float(max(scale_bits(sm.size[h]), sm.old[h]));
                const float inv = 1.f / s;
                uint8_t *dst = cache + sm.row[tok] * st.d_r + h * st.d_h;
#pragma unroll
                for (int k = 0; k < kUnits; ++k) {
                    int b_at;
                    const int at = unit_at<V, INTER, ROT>(piece * kUnits + k, rot_units, rot, pairs, b_at);
                    const float *w = x[i] + k * 2 * V;
                    uint32_t c[V]; // two codes each
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        c[e] = to_e4m3x2(w[2 * e] * inv, w[2 * e + 1] * inv);
                    if constexpr (V == 8) {
                        *reinterpret_cast<uint2 *>(dst + at) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                        *reinterpret_cast<uint2 *>(dst + at + b_at) = make_uint2(c[4] | c[5] << 16, c[6] | c[7] << 16);
                    } else if constexpr (V == 4) {
                        *reinterpret_cast<uint32_t *>(dst + at) = c[0] | c[1] << 16;
                        *reinterpret_cast<uint32_t *>(dst + at + b_at) = c[2] | c[3] << 16;
                    } else if constexpr (V == 2) {
                        *reinterpret_cast<uint16_t *>(dst + at) = static_cast<uint16_t>(c[0]);
                        *reinterpret_cast<uint16_t *>(dst + at + b_at) = static_cast<uint16_t>(c[1]);
                    } else {
                        dst[at] = static_cast<uint8_t>(c[0]);
                        dst[at + b_at] = static_cast<uint8_t>(c[0] >> 8);
                    }
                }
            }
        };

        __syncthreads(); // the last run's sizes have been read
        if (tid == 0)
            sm.fresh = 0;
        if (tid < f.div_group.d) {
            const float s = scale[tid];
            sm.size[tid] = 0u;
            sm.old[tid] = s > 0.f && s < -kNegInf ? __float_as_uint(s) : 0u;
        }
        // ---- the largest sizes of the run
        int n = find(start), total = n;
        const bool whole = block_of(start + n) != blk;
        load(start, n, true);
        if (!whole)
            while (n == f.chunk) {
                n = find(start + total);
                load(start + total, n, true);
                total += n;
            }
        __syncthreads();
        // ---- the scales: a block that begins drops the one it finds
        bool grows = false;
        if (tid < f.div_group.d) {
            if (sm.fresh)
                sm.old[tid] = 0u;
            const uint32_t need = scale_bits(sm.size[tid]);
            grows = sm.old[tid] && need > sm.old[tid];
            scale[tid] = __uint_as_float(max(need, sm.old[tid]));
        }
        if (__syncthreads_or(grows)) {
            // codes of the rows that the block holds (and of those about to be
            // written), eight at a time
            const int per = lpr * 2, units = sb * f.div_group.d * per;
            for (int i = tid; i < units; i += kRopeThreads) {
                const int r = i / per, u = i - r * per, row = fast_div(r, f.div_group), h = r - row * f.div_group.d;
                const uint32_t need = scale_bits(sm.size[h]), old = sm.old[h];
                if (need <= old || !old)
                    continue;
                const float ratio = __uint_as_float(old) / __uint_as_float(need);
                uint2 *at = reinterpret_cast<uint2 *>(cache + row * st.d_r + h * st.d_h + u * 8);
                const uint2 in = *at;
                uint32_t w[2] = {in.x, in.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 lo = from_e4m3x2(w[k] & 0xffffu), hi = from_e4m3x2(w[k] >> 16);
                    w[k] = to_e4m3x2(lo.x * ratio, lo.y * ratio) | to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
                }
                *at = make_uint2(w[0], w[1]);
            }
            __syncthreads();
        }
        // ---- the codes
        if (whole) {
            store(n);
        } else {
            for (int done = 0; done < total; done += n) {
                n = max(1, find(start + done));
                load(start + done, n, false);
                store(n);
            }
        }
    }
}

// Blocks of row y = 0 rotate q (where there is one); then K's groups of heads, then V's.
template <int V, bool INTER, bool ROT>
__global__ void __launch_bounds__(kRopeThreads, 2) append_fp8_kernel(const __grid_constant__ Fp8AppendParams f)
{
    __shared__ __align__(16) union {
        RunShared run;
        struct {
            float2 cs[kMaxAngles];
            int64_t src[kMaxTile], dst[kMaxTile];
        } rope;
    } sm;
    const int row = static_cast<int>(blockIdx.y) - f.rope.n_streams;
    if (row < 0) {
        rope_tile<__nv_bfloat16, V, INTER>(f.rope, f.rope.st[0], sm.rope.cs, sm.rope.src, sm.rope.dst);
        return;
    }
    if (blockIdx.x * f.tile >= f.rope.tokens)
        return;
    if (row < f.groups)
        append_runs<V, INTER, ROT>(f, f.k, row * f.div_group.d, sm.run);
    else
        append_runs<8, false, false>(f, f.v, (row - f.groups) * f.div_group.d, sm.run);
}

template <int V>
cudaError_t launch_append(Fp8AppendParams &f, bool interleaved, int blocks, cudaStream_t stream)
{
    const dim3 grid(blocks, f.rope.n_streams + 2 * f.groups);
    if (V == 8 && f.rope.pairs == 0)
        append_fp8_kernel<8, false, false><<<grid, kRopeThreads, 0, stream>>>(f);
    else if (interleaved)
        append_fp8_kernel<V, true, true><<<grid, kRopeThreads, 0, stream>>>(f);
    else
        append_fp8_kernel<V, false, true><<<grid, kRopeThreads, 0, stream>>>(f);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ reading back

constexpr int kReadThreads = 256;
constexpr int kReadUnits = 4; // units a thread has in flight

// A thread takes the codes of 16 bytes of output: neighbouring threads read and
// write neighbouring places.
template <class T>
__global__ void __launch_bounds__(kReadThreads) read_fp8_kernel(const __grid_constant__ Fp8ReadParams f)
{
    constexpr int E = 16 / sizeof(T);
    const Fp8ReadStream &st = f.st[blockIdx.y];
    const int t0 = blockIdx.x * f.tile, n_tok = min(f.tile, f.tokens - t0), units = n_tok * f.div_units.d;
    for (int i0 = threadIdx.x; i0 < units; i0 += kReadThreads * kReadUnits) {
        uint32_t w[kReadUnits][E / 4];
        float s[kReadUnits];
        int64_t to[kReadUnits];
#pragma unroll
        for (int k = 0; k < kReadUnits; ++k) {
            const int i = i0 + k * kReadThreads;
            to[k] = -1;
            if (i >= units)
                continue;
            const int tok = fast_div(i, f.div_units), rest = i - tok * f.div_units.d;
            const int h = rest >> f.head_shift, e = (rest & ((1 << f.head_shift) - 1)) * E;
            const int64_t slot = __ldg(f.slots + t0 + tok);
            if (slot < 0 || slot >= f.n_slots)
                continue;
            // slots and pages of 32 bits, as most caches have, divide faster
            const int64_t page = ((slot | f.page_rows) >> 32) == 0
                                     ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(f.page_rows)
                                     : slot / f.page_rows;
            const int64_t row = slot - page * f.page_rows;
            const uint8_t *src = st.cache + page * st.d_p + row * st.d_r + h * st.d_h + e;
#pragma unroll
            for (int q = 0; q < E / 4; ++q)
                w[k][q] = __ldg(reinterpret_cast<const uint32_t *>(src) + q);
            s[k] = __ldg(st.scale + page * st.s_p + (row >> f.block_shift) * st.s_b + h);
            to[k] = (t0 + tok) * st.o_t + h * st.o_h + e;
        }
#pragma unroll
        for (int k = 0; k < kReadUnits; ++k) {
            if (to[k] < 0)
                continue;
            float y[E];
#pragma unroll
            for (int q = 0; q < E / 2; ++q) {
                const float2 v = from_e4m3x2((q & 1 ? w[k][q / 2] >> 16 : w[k][q / 2]) & 0xffffu);
                y[2 * q] = v.x * s[k];
                y[2 * q + 1] = v.y * s[k];
            }
            T *dst = static_cast<T *>(st.out) + to[k];
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint4 *>(dst) = make_uint4(ptx::pack_bf16(y[0], y[1]), ptx::pack_bf16(y[2], y[3]),
                                                             ptx::pack_bf16(y[4], y[5]), ptx::pack_bf16(y[6], y[7]));
            else
                *reinterpret_cast<float4 *>(dst) = make_float4(y[0], y[1], y[2], y[3]);
        }
    }
}

} // namespace

cudaError_t launch_append_fp8(const Fp8AppendParams &params, bool interleaved, int sm_count, cudaStream_t stream)
{
    Fp8AppendParams f = params;
    RopeParams &p = f.rope;
    const int D = 16 << f.lane_shift;
    // pairs to a vector: the widest that divides the rotated pairs and the rest
    int V = 8;
    while (p.pairs % V || (D - p.rot) % (2 * V))
        V /= 2;
    // heads of a group: a divisor of their number, few enough that a whole block of
    // keys stays in registers
    const int rows = kRowsKept * (kRopeThreads >> f.lane_shift), sb = 1 << f.block_shift;
    int group = 1;
    for (int g = 2; g <= kRunHeads && g * sb <= rows; ++g)
        if (f.heads % g == 0)
            group = g;
    f.div_group = make_fastdiv(group);
    f.groups = f.heads / group;
    f.chunk = rows / group;
    if (p.pairs && f.chunk > kRunAngles / p.pairs)
        f.chunk = kRunAngles / p.pairs;
    f.chunk = f.chunk < sb ? f.chunk : sb;
    // tokens per thread block: a block of keys', as long as that fills the GPU
    f.tile = 1;
    while (f.tile < 32 && f.tile < sb && p.tokens / (2 * f.tile) >= 2 * sm_count)
        f.tile *= 2;
    int blocks = (p.tokens + f.tile - 1) / f.tile;
    if (p.n_streams) {
        const int q_blocks = rope_shape(p, V, sm_count);
        blocks = q_blocks > blocks ? q_blocks : blocks;
    }
    switch (V) {
    case 8: return launch_append<8>(f, interleaved, blocks, stream);
    case 4: return launch_append<4>(f, interleaved, blocks, stream);
    case 2: return launch_append<2>(f, interleaved, blocks, stream);
    default: return launch_append<1>(f, interleaved, blocks, stream);
    }
}

cudaError_t launch_read_fp8(const Fp8ReadParams &params, bool fp32, int sm_count, cudaStream_t stream)
{
    Fp8ReadParams f = params;
    // tokens per thread block: a few rounds of its threads, as long as that fills the GPU
    f.tile = 1;
    while (f.tile < 256 && int64_t(f.tile) * f.div_units.d < 2 * kReadThreads * kReadUnits &&
           f.tokens / (2 * f.tile) >= 4 * sm_count)
        f.tile *= 2;
    const dim3 grid((f.tokens + f.tile - 1) / f.tile, f.n_streams);
    if (fp32)
        read_fp8_kernel<float><<<grid, kReadThreads, 0, stream>>>(f);
    else
        read_fp8_kernel<__nv_bfloat16><<<grid, kReadThreads, 0, stream>>>(f);
    return cudaGetLastError();
}

} // namespace fl
