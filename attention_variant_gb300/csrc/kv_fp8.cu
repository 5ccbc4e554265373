// kv_fp8.cu -- new keys and values into a paged cache of e4m3 codes, rotated on
// the way, and tokens of such a cache read back.
//
//   code = rn(x / s),  s the scale of the row's block of keys and head
//
// s is the smallest power of two that 448 s holds every finite |x| of the block,
// at least 2^-100: then x / s is exact, and a scale that grows leaves codes c -> rn(c
// s_old / s), which rounds subnormals alone.  So the codes of a block hardly depend on how
// its tokens were split over calls, and its scale not at all.  (A scale found may be no power
// of two: quotients and products are rounded once then, too, by the exact sign of what is left.)
//
// The tokens of a block that a call brings are neighbours but for skipped ones (fl_kv_plan lists
// them so): a run, with the skipped ones inside and behind it.  A thread block takes the runs that
// begin in its window of tokens, as many at a time as fit, for a group of heads: each thread keeps
// its 16 elements of up to four (token, head) rows in registers from the maximum (over the lanes of
// a row, then in shared memory) to the codes (as bf16, and rotates them twice: kept rotated, in
// fp32, they left two blocks to a SM).  A run too long for that is read and rotated twice, the
// second time out of L2.
//
// Bound by HBM in part, and by the rotation: 11,810 tokens of 16 + 2 + 2 heads of 128 take 35.8 us
// (3210 GB/s of 6794; q's rotation, a kernel of its own beside, is 80% of the bytes);
// 64 single tokens 5.1 us, the launch and one chain of loads.  Reading 79,000 tokens back
// into bf16 35.8 us, 6070 GB/s.
#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "e4m3.cuh"
#include "rope.cuh"

namespace fl {
namespace {

constexpr int kRowsKept = 4;      // (token, head) rows a thread keeps
constexpr int kRunRows = 256;     // of a thread block, at most
constexpr int kRunAngles = 4096;  // tokens of a chunk times pairs
constexpr int kRunHeads = 16;     // heads of a group, at most

struct RunShared {
    float2 cs[kRunAngles];
    int64_t place[kRunRows];      // of each token of the chunk: its row in the cache, or -1
    int64_t block[kRunRows];      // of each run: its first row in the cache
    int64_t scale[kRunRows];      // and its scales
    int32_t pos[kRunRows];        // position of each token
    uint32_t size[kRunRows];      // of each run and head: the largest |x|, as bits
    uint32_t old[kRunRows];       // and the scale before
    uint8_t run[kRunRows], fresh[kRunRows]; // run of each token; the run has its block's first row
    int leaders[kRopeThreads / 32];
    int end, last;
    int64_t last_block;
};

// Two quotients x / m to codes, for 1 <= m < 2, rounded once: where x times 1 / m, off by less than
// 4 of its last places, is that near a number of 8 bits -- the borders between codes are
// some of these --, the sign of x - g m, exact, says on which side x / m lies.
__device__ __noinline__ uint32_t quotients_to_e4m3x2(float x0, float x1, float m)
{
    const float inv = 1.f / m, x[2] = {x0, x1};
    float y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        y[i] = x[i] * inv;
        const uint32_t b = __float_as_uint(y[i]), g = (b + 0x8000u) & 0xffff0000u;
        if (fabsf(y[i]) < 1024.f && b - g + 4u <= 8u) { // (past 448 anything is 448; NaN stays NaN)
            const float r = fmaf(-__uint_as_float(g), m, x[i]);
            y[i] = __uint_as_float(r == 0.f ? g : (r > 0.f) == (x[i] > 0.f) ? g + 1u : g - 1u);
        }
    }
    return to_e4m3x2(y[0], y[1]);
}

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

// The runs that begin among the window's tokens, for heads h0 .. h0 + group - 1.
template <int V, bool INTER, bool ROT>
__device__ __forceinline__ void append_runs(const Fp8AppendParams &f, const Fp8Stream &st, int h0, RunShared &sm)
{
    constexpr int kUnits = 8 / V; // of a thread's 16 elements
    const RopeParams &p = f.rope;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = f.div_group.d;
    const int lpr = 1 << f.lane_shift, piece = tid & (lpr - 1), y = tid >> f.lane_shift, rp = kRopeThreads >> f.lane_shift;
    const int rot = ROT ? p.rot : 0, pairs = ROT ? p.pairs : 0, rot_units = pairs / V;
    const int t0 = blockIdx.x * f.tile, t1 = min(t0 + f.tile, p.tokens), sb = 1 << f.block_shift;
    auto block_of = [&](int t) { // -1: skipped
        const int64_t slot = t >= 0 && t < p.tokens ? __ldg(p.slots + t) : -1;
        return slot < 0 || slot >= p.n_slots ? int64_t(-1) : slot >> f.block_shift;
    };
    // a block's first row in the cache and its scales
    auto locate = [&](int64_t blk, int64_t &row, int64_t &scale) {
        const int64_t first = blk << f.block_shift;
        // slots and pages of 32 bits, as most caches have, divide faster
        const int64_t page = ((first | p.page_rows) >> 32) == 0
                                 ? static_cast<uint32_t>(first) / static_cast<uint32_t>(p.page_rows)
                                 : first / p.page_rows;
        const int64_t in = first - page * p.page_rows;
        row = page * st.d_p + in * st.d_r + h0 * st.d_h;
        scale = page * st.s_p + (in >> f.block_shift) * st.s_b + h0;
    };
    // a token of the chunk
    auto place_token = [&](int i, int t, int run, int64_t row, bool position) {
        const int in = static_cast<int>(__ldg(p.slots + t) & (sb - 1));
        sm.place[i] = row + in * st.d_r;
        if (ROT && position)
            sm.pos[i] = __ldg(p.positions + t);
        sm.run[i] = static_cast<uint8_t>(run);
        if (in == 0)
            sm.fresh[run] = 1;
    };
    // a thread meets one frequency where the pairs divide the threads; frequencies are
    // constants, which the lanes of a warp fetch one after another
    int turn_i = 0;
    uint64_t turn = 0;
    if constexpr (ROT) {
        turn_i = tid - fast_div(tid, p.div_pairs) * pairs;
        turn = p.turns[turn_i];
    }
    auto angles = [&](int n) {
        if constexpr (ROT) {
            for (int e = tid; e < n * pairs; e += kRopeThreads) {
                const int tl = fast_div(e, p.div_pairs), i = e - tl * pairs;
                if (i != turn_i) {
                    turn_i = i;
                    turn = p.turns[i];
                }
                float2 cs = turn_cos_sin(static_cast<uint64_t>(p.offset + sm.pos[tl]) * turn);
                cs.x *= p.magnitude;
                cs.y *= p.magnitude;
                sm.cs[tl * pairs + angle_at<V>(i, rot_units)] = cs;
            }
        }
    };
    uint32_t raw[kRowsKept][8]; // this thread's elements of its rows: per unit V of a, V of b
    auto load = [&](int c0, int n) {
#pragma unroll
        for (int i = 0; i < kRowsKept; ++i) {
            const int r = y + i * rp, tok = fast_div(r, f.div_group), h = r - tok * group;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                raw[i][e] = 0u;
            if (tok >= n || sm.place[tok] < 0)
                continue;
            const __nv_bfloat16 *src = st.src + static_cast<int64_t>(c0 + tok) * st.s_s + (h0 + h) * st.s_h;
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                int b_at;
                const int at = unit_at<V, INTER, ROT>(piece * kUnits + k, rot_units, rot, pairs, b_at);
                if constexpr (V == 1) {
                    const uint16_t *w = reinterpret_cast<const uint16_t *>(src);
                    raw[i][k] = w[at] | static_cast<uint32_t>(w[at + b_at]) << 16;
                } else {
                    using W = Vec<uint32_t, V / 2 == 0 ? 1 : V / 2>;
                    const W a = *reinterpret_cast<const W *>(src + at), b = *reinterpret_cast<const W *>(src + at + b_at);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        raw[i][k * V + e] = a.e[e];
                        raw[i][k * V + V / 2 + e] = b.e[e];
                    }
                }
            }
        }
    };
    // Row i's elements in fp32, rotated, and the largest size among them; what is
    // infinite is not a number.
    auto expand = [&](int i, int tok, float (&x)[16]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[2 * e] = __uint_as_float(raw[i][e] << 16);
            x[2 * e + 1] = __uint_as_float(raw[i][e] & 0xffff0000u);
        }
        if constexpr (ROT) {
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                const int u = piece * kUnits + k;
                float *w = x + k * 2 * V;
                if (u < rot_units) {
                    const float2 *cs = sm.cs + tok * pairs + u * (V == 1 ? 1 : 2);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float2 c = V <= 2 ? cs[e] : cs[(e / 2) * rot_units * 2 + e % 2];
                        float &ra = INTER ? w[2 * e] : w[e], &rb = INTER ? w[2 * e + 1] : w[V + e];
                        const float xa = ra, xb = rb;
                        ra = xa * c.x - xb * c.y;
                        rb = xa * c.y + xb * c.x;
                    }
                }
            }
        }
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            m = fmaxf(m, fabsf(x[e]));
        if (m == -kNegInf) {
            m = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (fabsf(x[e]) == -kNegInf)
                    x[e] = __uint_as_float(0x7fffffffu);
                else
                    m = fmaxf(m, fabsf(x[e]));
            }
        }
        return m;
    };
    auto measure = [&](int n) {
#pragma unroll
        for (int i = 0; i < kRowsKept; ++i) {
            const int r = y + i * rp, tok = fast_div(r, f.div_group), h = r - tok * group;
            if (y - lane / lpr + i * rp >= n * group)
                break; // no row of the warp's is in the chunk
            float x[16];
            uint32_t top = __float_as_uint(expand(i, tok < n ? tok : 0, x));
            for (int d = lpr / 2; d; d >>= 1)
                top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (tok < n && piece == 0 && top)
                atomicMax(&sm.size[sm.run[tok] * group + h], top);
        }
    };
    auto store = [&](int n) {
#pragma unroll
        for (int i = 0; i < kRowsKept; ++i) {
            const int r = y + i * rp, tok = fast_div(r, f.div_group), h = r - tok * group;
            if (tok >= n || sm.place[tok] < 0)
                continue;
            float x[16];
            expand(i, tok, x);
            const int at_run = sm.run[tok] * group + h;
            const float s = __uint_as_float(max(scale_bits(sm.size[at_run]), sm.old[at_run]));
            // s = m times a power of two; m is 1 but for scales from elsewhere
            const float m = __uint_as_float((__float_as_uint(s) & 0x7fffffu) | 0x3f800000u);
            const float inv = 1.f / __uint_as_float(__float_as_uint(s) & 0x7f800000u);
            uint8_t *dst = st.cache + sm.place[tok] + h * st.d_h;
            uint32_t codes[8]; // two each
            if (m == 1.f) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    codes[e] = to_e4m3x2(x[2 * e] * inv, x[2 * e + 1] * inv);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    codes[e] = quotients_to_e4m3x2(x[2 * e] * inv, x[2 * e + 1] * inv, m);
            }
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                int b_at;
                const int at = unit_at<V, INTER, ROT>(piece * kUnits + k, rot_units, rot, pairs, b_at);
                const uint32_t *c = codes + k * V;
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

    // Is the first token from u on that is not skipped one of block blk?  All threads, 16 tokens
    // each at a time.  (64 tokens and 960 of padding take 9.0 us; 8.5 where a run ended at a skipped slot.)
    auto goes_on = [&](int u, int64_t blk) {
        constexpr int kAhead = 16;
        for (; u < p.tokens; u += kAhead * kRopeThreads) {
            const int64_t here = block_of(u);
            if (here >= 0)
                return here == blk;
            int at = INT32_MAX;
#pragma unroll
            for (int i = kAhead - 1; i >= 0; --i)
                at = block_of(u + i * kRopeThreads + tid) >= 0 ? u + i * kRopeThreads + tid : at;
            if (!__syncthreads_or(at < INT32_MAX))
                continue;
            if (tid == 0)
                sm.end = INT32_MAX;
            __syncthreads();
            if (at < INT32_MAX)
                atomicMin(&sm.end, at);
            __syncthreads();
            at = sm.end;
            return block_of(at) == blk;
        }
        return false;
    };

    for (int s = t0; s < t1;) {
        // ---- the chunk: tokens s .. s + n - 1, whole runs but the one that began before the
        // window, or (longer) the beginning of a run that does not fit
        __syncthreads(); // the last chunk's have been read
        if (tid == 0) {
            sm.end = f.chunk;
            sm.last = -1;
        }
        const int t = s + tid;
        const int64_t mine = tid < f.chunk ? block_of(t) : -1;
        if (ROT && tid < f.chunk)
            sm.pos[tid] = t < p.tokens ? __ldg(p.positions + t) : 0;
        // the block of the last token before that is not skipped
        int64_t before = block_of(t - 1);
        for (uint32_t todo = __ballot_sync(0xffffffffu, mine >= 0 && before < 0); todo; todo &= todo - 1) {
            const int of = __ffs(todo) - 1;
            int64_t found = -1;
            for (int u = s + warp * 32 + of - 2 - lane;; u -= 32) { // 32 tokens at a time
                const int64_t b = block_of(u);
                const uint32_t hit = __ballot_sync(0xffffffffu, b >= 0 || u < 0);
                if (hit) {
                    found = __shfl_sync(0xffffffffu, b, __ffs(hit) - 1);
                    break;
                }
            }
            if (lane == of)
                before = found;
        }
        const bool leader = mine >= 0 && mine != before;
        const uint32_t ballot = __ballot_sync(0xffffffffu, leader);
        if (lane == 0)
            sm.leaders[warp] = __popc(ballot);
        sm.fresh[tid] = 0;
        __syncthreads();
        int run = __popc(ballot & (0xffffffffu >> (31 - lane))) - 1; // of this token; -1: began before
#pragma unroll
        for (int w = 0; w < kRopeThreads / 32; ++w)
            run += w < warp ? sm.leaders[w] : 0;
        if (tid < f.chunk && (t >= p.tokens || (leader && t >= t1) || (run < 0 && t >= t1)))
            atomicMin(&sm.end, tid); // the next window's, or past the last
        __syncthreads();
        int n = sm.end;
        if (leader && tid < n)
            atomicMax(&sm.last, tid);
        __syncthreads();
        const int last = sm.last;
        bool go_long = false;
        if (n == f.chunk && last >= 0) { // the last run may go on past the chunk
            if (tid == last)
                sm.last_block = mine;
            __syncthreads();
            if (goes_on(s + n, sm.last_block)) {
                go_long = last == 0;
                n = go_long ? n : last;
            }
        }
        if (n == 0)
            break;
        if (tid < n) {
            sm.place[tid] = -1;
            sm.run[tid] = 0;
        }
        int64_t row = 0, scale = 0;
        if (tid < n && mine >= 0 && run >= 0) {
            locate(mine, row, scale);
            if (leader) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(st.scale + scale));
                sm.block[run] = row;
                sm.scale[run] = scale;
            }
            place_token(tid, t, run, row, false);
        }
        int runs = 0;
        {
            const uint32_t in = __ballot_sync(0xffffffffu, leader && tid < n);
            __syncthreads();
            if (lane == 0)
                sm.leaders[warp] = __popc(in);
            load(s, n);
            angles(n);
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kRopeThreads / 32; ++w)
                runs += sm.leaders[w];
        }
        for (int i = tid; i < runs * group; i += kRopeThreads) {
            const int r = fast_div(i, f.div_group);
            const float old = st.scale[sm.scale[r] + i - r * group];
            sm.size[i] = 0u;
            sm.old[i] = old > 0.f && old < -kNegInf ? __float_as_uint(old) : 0u;
        }
        __syncthreads();
        // ---- the largest sizes of each run
        measure(n);
        int total = n;
        if (go_long) {
            const int64_t blk = block_of(s);
            const int64_t block_row = sm.block[0];
            for (int more = n; more == f.chunk && goes_on(s + total, blk); total += more) {
                __syncthreads();
                if (tid == 0)
                    sm.end = f.chunk;
                __syncthreads();
                if (tid < f.chunk) {
                    const int x = s + total + tid;
                    const int64_t b = block_of(x);
                    if (x >= p.tokens || (b >= 0 && b != blk))
                        atomicMin(&sm.end, tid);
                    sm.place[tid] = -1;
                    if (b == blk)
                        place_token(tid, x, 0, block_row, true);
                }
                __syncthreads();
                more = sm.end;
                load(s + total, more);
                angles(more);
                __syncthreads();
                measure(more);
            }
        }
        __syncthreads();
        // ---- the scales: a block that begins drops the one it finds
        bool grows = false;
        for (int i = tid; i < runs * group; i += kRopeThreads) {
            const int r = fast_div(i, f.div_group);
            if (sm.fresh[r])
                sm.old[i] = 0u;
            const uint32_t need = scale_bits(sm.size[i]);
            grows |= sm.old[i] && need > sm.old[i];
            st.scale[sm.scale[r] + i - r * group] = __uint_as_float(max(need, sm.old[i]));
        }
        if (__syncthreads_or(grows)) {
            // codes of the rows that the blocks hold (and of those about to be
            // written), eight at a time
            const int per = lpr * 2;
            for (int i = 0; i < runs * group; ++i) {
                const uint32_t need = scale_bits(sm.size[i]), old = sm.old[i];
                if (need <= old || !old)
                    continue;
                const int r = fast_div(i, f.div_group);
                const float ratio = __uint_as_float(old) / __uint_as_float(need);
                uint8_t *const block = st.cache + sm.block[r] + (i - r * group) * st.d_h;
                for (int j = tid; j < sb * per; j += kRopeThreads) {
                    const int in = j / per;
                    uint2 *at = reinterpret_cast<uint2 *>(block + in * st.d_r + (j - in * per) * 8);
                    const uint2 was = *at;
                    uint32_t w[2] = {was.x, was.y};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 lo = from_e4m3x2(w[k] & 0xffffu), hi = from_e4m3x2(w[k] >> 16);
                        w[k] = to_e4m3x2(times_to_odd(lo.x, ratio), times_to_odd(lo.y, ratio)) |
                               to_e4m3x2(times_to_odd(hi.x, ratio), times_to_odd(hi.y, ratio)) << 16;
                    }
                    *at = make_uint2(w[0], w[1]);
                }
            }
            __syncthreads();
        }
        // ---- the codes
        if (!go_long) {
            store(n);
        } else {
            const int64_t blk = block_of(s), block_row = sm.block[0];
            for (int done = 0, more; done < total; done += more) {
                __syncthreads();
                more = min(f.chunk, total - done);
                if (tid < more) {
                    sm.place[tid] = -1;
                    if (block_of(s + done + tid) == blk)
                        place_token(tid, s + done + tid, 0, block_row, true);
                }
                __syncthreads();
                load(s + done, more);
                angles(more);
                __syncthreads();
                store(more);
            }
        }
        s += total;
    }
}

// Blocks of the first row rotate q, where it comes along; then K's groups of heads, then V's.
template <int V, bool INTER, bool ROT>
__global__ void __launch_bounds__(kRopeThreads, 3) append_fp8_kernel(const __grid_constant__ Fp8AppendParams f)
{
    __shared__ __align__(16) union {
        RunShared run;
        struct {
            float2 cs[kMaxAngles];
            int64_t src[kMaxTile], dst[kMaxTile];
        } rope;
    } sm;
    const int row = static_cast<int>(blockIdx.y) - f.q_rows;
    if (row < 0)
        rope_tile<__nv_bfloat16, V, INTER>(f.rope, f.rope.st[0], sm.rope.cs, sm.rope.src, sm.rope.dst);
    else if (blockIdx.x * f.tile < f.rope.tokens) {
        if (row < f.groups)
            append_runs<V, INTER, ROT>(f, f.k, row * f.div_group.d, sm.run);
        else
            append_runs<8, false, false>(f, f.v, (row - f.groups) * f.div_group.d, sm.run);
    }
    ptx::wait_dependency(); // q's own kernel, which may still run, has to end before this one
}

// q by itself, eight blocks to a SM.
template <int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 8) append_q_kernel(const __grid_constant__ Fp8AppendParams f)
{
    __shared__ __align__(16) float2 s_cs[kMaxAngles];
    __shared__ int64_t s_src[kMaxTile], s_dst[kMaxTile];
    ptx::launch_dependents();
    rope_tile<__nv_bfloat16, V, INTER>(f.rope, f.rope.st[0], s_cs, s_src, s_dst);
}

template <int V, bool INTER, bool ROT>
cudaError_t launch_append(Fp8AppendParams &f, int sm_count, cudaStream_t stream)
{
    int blocks = (f.rope.tokens + f.tile - 1) / f.tile;
    cudaLaunchAttribute attr{};
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    if (f.rope.n_streams) {
        // where q has more blocks than the two of this kernel that a SM holds carry, they get a
        // kernel of their own (11,810 tokens of 16 heads of 128: 50 -> 36 us), else a
        // launch is saved
        const int q_blocks = rope_shape(f.rope, V, sm_count);
        if (q_blocks > 4 * sm_count) {
            append_q_kernel<V, INTER><<<q_blocks, kRopeThreads, 0, stream>>>(f);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess)
                return e;
            attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr.val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
        } else {
            f.q_rows = 1;
            blocks = q_blocks > blocks ? q_blocks : blocks;
        }
    }
    cfg.gridDim = dim3(blocks, f.q_rows + 2 * f.groups);
    return cudaLaunchKernelEx(&cfg, append_fp8_kernel<V, INTER, ROT>, f);
}

template <int V>
cudaError_t launch_append_vec(Fp8AppendParams &f, bool interleaved, int sm_count, cudaStream_t stream)
{
    if (V == 8 && f.rope.pairs == 0)
        return launch_append<8, false, false>(f, sm_count, stream);
    return interleaved ? launch_append<V, true, true>(f, sm_count, stream)
                       : launch_append<V, false, true>(f, sm_count, stream);
}

// ------------------------------------------------------------------ reading back

constexpr int kReadThreads = 256;
constexpr int kReadUnits = 4; // tokens a thread has in flight
constexpr int kReadTile = 64;

// A thread takes the codes of 16 bytes of output, at one place of the heads for
// several tokens; neighbouring threads read and write neighbouring places.  What a token's
// slot says is worked out once, for all of its heads.
template <class T>
__global__ void __launch_bounds__(kReadThreads) read_fp8_kernel(const __grid_constant__ Fp8ReadParams f)
{
    constexpr int E = 16 / sizeof(T);
    __shared__ int64_t s_row[kReadTile], s_scale[kReadTile]; // of each token, in the cache; < 0: skipped
    const Fp8ReadStream &st = f.st[blockIdx.y];
    const int tid = threadIdx.x, t0 = blockIdx.x * f.tile, n_tok = min(f.tile, f.tokens - t0);
    if (tid < n_tok) {
        const int64_t slot = __ldg(f.slots + t0 + tid);
        int64_t row = -1, scale = 0;
        if (slot >= 0 && slot < f.n_slots) {
            // slots and pages of 32 bits, as most caches have, divide faster
            const int64_t page = ((slot | f.page_rows) >> 32) == 0
                                     ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(f.page_rows)
                                     : slot / f.page_rows;
            const int64_t in = slot - page * f.page_rows;
            row = page * st.d_p + in * st.d_r;
            scale = page * st.s_p + (in >> f.block_shift) * st.s_b;
        }
        s_row[tid] = row;
        s_scale[tid] = scale;
    }
    __syncthreads();
    const int y = fast_div(tid, f.div_units), x = tid - y * f.div_units.d;
    if (y >= f.uy)
        return;
    for (int u = x; u < f.units; u += f.div_units.d) {
        const int h = u >> f.head_shift, e = (u & ((1 << f.head_shift) - 1)) * E;
        const uint8_t *src = st.cache + h * st.d_h + e;
        const float *scale = st.scale + h;
        T *out = static_cast<T *>(st.out) + t0 * st.o_t + h * st.o_h + e;
        for (int t = y; t < n_tok; t += kReadUnits * f.uy) {
            uint32_t w[kReadUnits][E / 4];
            float s[kReadUnits];
#pragma unroll
            for (int k = 0; k < kReadUnits; ++k) {
                const int tok = t + k * f.uy;
                const int64_t row = tok < n_tok ? s_row[tok] : -1;
                if constexpr (sizeof(T) == 2)
                    s[k] = 0.f;
                if (row < 0)
                    continue;
                if constexpr (E == 8) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + row));
                    w[k][0] = v.x;
                    w[k][1] = v.y;
                } else {
                    w[k][0] = __ldg(reinterpret_cast<const uint32_t *>(src + row));
                }
                s[k] = __ldg(scale + s_scale[tok]);
            }
            // a product of up to 28 bits; into bf16 only exact ones may go by way of fp32
            uint32_t rest = 0;
#pragma unroll
            for (int k = 0; k < (sizeof(T) == 2 ? kReadUnits : 0); ++k)
                rest |= __float_as_uint(s[k]) & 0x7fffffu;
            auto write = [&](auto once) {
                constexpr bool ONCE = decltype(once)::value;
#pragma unroll
                for (int k = 0; k < kReadUnits; ++k) {
                    const int tok = t + k * f.uy;
                    if (tok >= n_tok || s_row[tok] < 0)
                        continue;
                    float v[E];
#pragma unroll
                    for (int q = 0; q < E / 2; ++q) {
                        const float2 c = from_e4m3x2((q & 1 ? w[k][q / 2] >> 16 : w[k][q / 2]) & 0xffffu);
                        v[2 * q] = ONCE ? times_to_odd(c.x, s[k]) : c.x * s[k];
                        v[2 * q + 1] = ONCE ? times_to_odd(c.y, s[k]) : c.y * s[k];
                    }
                    T *dst = out + tok * st.o_t;
                    if constexpr (sizeof(T) == 2)
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(ptx::pack_bf16(v[0], v[1]), ptx::pack_bf16(v[2], v[3]),
                                                                     ptx::pack_bf16(v[4], v[5]), ptx::pack_bf16(v[6], v[7]));
                    else
                        *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                }
            };
            if (rest == 0)
                write(std::false_type{});
            else
                write(std::true_type{});
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
    // keys stays in registers (of few tokens, which are hardly all of one block, 32 keys:
    // 64 single tokens of 8 heads, scales by 256 keys: 12.8 us with a head to a group, 4.9
    // with all)
    const int rows = kRowsKept * (kRopeThreads >> f.lane_shift), sb = 1 << f.block_shift;
    const int keys = p.tokens <= 2 * sm_count && sb > 32 ? 32 : sb;
    int group = 1;
    for (int g = 2; g <= kRunHeads && g * keys <= rows; ++g)
        if (f.heads % g == 0)
            group = g;
    f.div_group = make_fastdiv(group);
    f.groups = f.heads / group;
    f.chunk = rows / group;
    if (p.pairs && f.chunk > kRunAngles / p.pairs)
        f.chunk = kRunAngles / p.pairs;
    // tokens of a window: those of a chunk, as long as that fills the GPU
    f.tile = 1;
    while (2 * f.tile <= f.chunk && p.tokens / (2 * f.tile) * 2 * f.groups >= 2 * sm_count)
        f.tile *= 2;
    switch (V) {
    case 8: return launch_append_vec<8>(f, interleaved, sm_count, stream);
    case 4: return launch_append_vec<4>(f, interleaved, sm_count, stream);
    case 2: return launch_append_vec<2>(f, interleaved, sm_count, stream);
    default: return launch_append_vec<1>(f, interleaved, sm_count, stream);
    }
}

cudaError_t launch_read_fp8(const Fp8ReadParams &params, bool fp32, int sm_count, cudaStream_t stream)
{
    Fp8ReadParams f = params;
    const int units = f.units < kReadThreads ? f.units : kReadThreads;
    f.div_units = make_fastdiv(units);
    f.uy = kReadThreads / units;
    // tokens per thread block: two rounds of its threads, as long as that fills the GPU
    f.tile = 1;
    while (f.tile < kReadTile && f.tile < 2 * kReadUnits * f.uy && f.tokens / (2 * f.tile) >= 4 * sm_count)
        f.tile *= 2;
    const dim3 grid((f.tokens + f.tile - 1) / f.tile, f.n_streams);
    if (fp32)
        read_fp8_kernel<float><<<grid, kReadThreads, 0, stream>>>(f);
    else
        read_fp8_kernel<__nv_bfloat16><<<grid, kReadThreads, 0, stream>>>(f);
    return cudaGetLastError();
}

} // namespace fl
