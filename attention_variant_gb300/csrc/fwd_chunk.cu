// fwd_chunk.cu -- attention of ragged chunks of new tokens over the cache
// that holds them (serving: prompts, parts of prompts and single tokens in
// one call), paged or contiguous.
//
// The plain form: a warp per (token, head), its lanes sharing the head
// dimension, an online softmax over the keys one by one.
#include <cuda_bf16.h>
#include <cstdint>

#include "common.cuh"
#include "launch.h"

namespace fl {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) chunk_kernel(const ChunkParams p)
{
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int t = static_cast<int>(w / p.Hq), h = static_cast<int>(w % p.Hq);
    if (t >= p.T)
        return;
    int lo = 0, hi = p.batch - 1; // the last request that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.cu_q + mid) <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int b = lo, c0 = max(0, __ldg(p.cu_q + b)), c1 = min(p.T, __ldg(p.cu_q + b + 1));
    if (t < c0 || t >= c1)
        return; // a row of no request
    const int L = max(0, min(__ldg(p.kv_lens + b), p.max_kv));
    const int pos = L - (c1 - c0) + (t - c0);
    const int j1 = p.causal ? min(L, pos + 1) : L;
    const int j0 = p.window ? max(0, pos - p.window + 1) : 0;
    constexpr int E = D / 32;
    const int hk = h / p.G;
    float q[E], o[E], m = kNegInf, l = 0.f;
    const __nv_bfloat16 *qp = p.q + t * p.q_st + h * p.q_sh + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(qp[e]);
        o[e] = 0.f;
    }
    for (int j = j0; j < j1; ++j) {
        int64_t page = b, row = j;
        if (p.page_shift >= 0) {
            page = __ldg(p.block_table + b * p.bt_stride + (j >> p.page_shift));
            row = j & ((1 << p.page_shift) - 1);
        }
        const bool in = page >= 0 && page < p.n_pages;
        const __nv_bfloat16 *kp = p.k + page * p.k_sp + row * p.k_sr + hk * p.k_sh + lane * E;
        const __nv_bfloat16 *vp = p.v + page * p.v_sp + row * p.v_sr + hk * p.v_sh + lane * E;
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            z = fmaf(q[e], in ? __bfloat162float(kp[e]) : 0.f, z);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            z += __shfl_xor_sync(0xffffffffu, z, d);
        z *= p.scale;
        if (p.score_mod == MOD_SOFTCAP)
            z = p.softcap * tanhf(z / p.softcap);
        const float m1 = fmaxf(m, z), a = expf(m - m1), x = expf(z - m1);
        m = m1;
        l = l * a + x;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * a + x * (in ? __bfloat162float(vp[e]) : 0.f);
    }
    __nv_bfloat16 *op = p.out + t * p.o_st + h * p.o_sh + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e)
        op[e] = __float2bfloat16(l > 0.f ? o[e] / l : 0.f);
    if (lane == 0 && p.lse)
        p.lse[h * p.l_sh + t] = l > 0.f ? m + logf(l) : kNegInf;
}

} // namespace

cudaError_t launch_chunk(const ChunkParams &p, cudaStream_t stream)
{
    const int64_t blocks = (int64_t(p.T) * p.Hq + 3) / 4;
    if (p.head_dim == 64)
        chunk_kernel<64><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
    else
        chunk_kernel<128><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

} // namespace fl
