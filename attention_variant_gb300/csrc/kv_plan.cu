// kv_plan.cu -- the book-keeping of a serving step on the GPU: first tokens
// of the requests (a sum over their lengths), new cache lengths, the position
// and cache slot of every new token, and the pages the step adds to the block
// table.
//
// Every block sums over all requests itself (kSeqs at a time, lengths and new
// pages packed in one 64-bit scan), which costs a few hundred cycles a kSeqs
// and spares a second launch; it then handles its own kTokens tokens, which
// find their request by bisection in shared memory.  A page that the step
// adds starts with a new token, and that token writes its table entry: no
// thread loops over pages, and entries that are read (pages held before
// the step) are never written.  Only where tokens are not listed (there are more
// than max_tokens) are the pages that these begin counted up and shared out.
#include <cstdint>

#include "common.cuh"
#include "fl_attn.h"
#include "launch.h"

namespace fl {
namespace {

constexpr int kThreads = 1024;
constexpr int kSeqs = 1024;   // requests per scan
constexpr int kTokens = 1024; // tokens per block

// Inclusive sum over the block (of packed pairs, low: tokens, high: pages).
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d)
            x += y;
    }
    if (lane == 31)
        s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        uint64_t w = s_warp[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d)
                w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    return x + (warp ? s_warp[warp - 1] : 0);
}

// The requests of a scan, by thread.
struct PlanShared {
    uint64_t warp[32];
    int cu[kSeqs + 1];   // first token of each, then their end
    int kv[kSeqs];
    int first[kSeqs];    // place of its first new page on the free list
    int64_t rest[kSeqs]; // new pages that no listed token begins, summed up
    int page[kSeqs];     // the first of them
};

// Table entries of the new pages that no listed token begins, of a scan some of
// whose tokens are not listed; this thread's request has n new tokens, kv keys on
// `held` pages and then `need`.  Returns error bits.  (A function of its own: in the
// kernel's body it cost steps that list every token 0.2 of 2.7 us.)
__device__ __noinline__ uint32_t unlisted_pages(const KvPlanParams &p, PlanShared &sm, int b0, int n, int kv, int held,
                                                int need)
{
    const int tid = threadIdx.x, page_mask = (1 << p.page_shift) - 1, stride = p.bt_stride;
    uint32_t err = n && need > stride ? FL_DEVERR_PAGES : 0;
    // (64 bits: lengths without meaning stay inside the table)
    const int64_t left = static_cast<int64_t>(p.max_tokens) - sm.cu[tid];
    const int64_t from = left > 0 ? (left + kv + page_mask) >> p.page_shift : 0;
    const int64_t at = from > held ? from : held, to = need < stride ? need : stride;
    const int64_t mine = b0 + tid < p.batch && to > at ? to - at : 0;
    sm.rest[tid] = static_cast<int64_t>(block_scan(static_cast<uint64_t>(mine), sm.warp));
    sm.page[tid] = static_cast<int>(at < stride ? at : stride);
    __syncthreads();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + tid; i < sm.rest[kSeqs - 1]; i += step) {
        int lo = 0, hi = kSeqs - 1; // the first request whose sum is past i
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sm.rest[mid] > i)
                hi = mid;
            else
                lo = mid + 1;
        }
        const int page = sm.page[lo] + static_cast<int>(i - (lo ? sm.rest[lo - 1] : 0));
        const int had = static_cast<int>((static_cast<uint32_t>(sm.kv[lo]) + page_mask) >> p.page_shift);
        const int on_list = sm.first[lo] + page - had;
        const int id = on_list >= 0 && on_list < p.n_free ? __ldg(p.free_pages + on_list) : -1;
        p.block_table[static_cast<int64_t>(b0 + lo) * stride + page] = id;
        if (id < 0)
            err |= FL_DEVERR_PAGES;
    }
    return err;
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const __grid_constant__ KvPlanParams p)
{
    __shared__ PlanShared sm;
    const int tid = threadIdx.x;
    const int t = blockIdx.x * kTokens + tid;
    const int page_mask = (1 << p.page_shift) - 1;
    const int head = __ldg(p.free_head);
    uint32_t err = 0;
    int tokens = 0, pages = 0; // of the requests before this scan
    for (int b0 = 0; b0 < p.batch; b0 += kSeqs) {
        const int b = b0 + tid;
        int n = 0, kv = 0;
        if (b < p.batch) {
            n = max(0, __ldg(p.q_lens + b));
            kv = max(0, __ldg(p.kv_lens + b));
        }
        const uint32_t held = (static_cast<uint32_t>(kv) + page_mask) >> p.page_shift;
        const uint32_t fresh = ((static_cast<uint32_t>(kv) + n + page_mask) >> p.page_shift) - held;
        const uint64_t sum = block_scan((static_cast<uint64_t>(fresh) << 32) | static_cast<uint32_t>(n), sm.warp);
        const int end = tokens + static_cast<int>(static_cast<uint32_t>(sum));
        const int last_page = pages + static_cast<int>(sum >> 32);
        const int pages_end = pages + static_cast<int>(sm.warp[31] >> 32);
        sm.cu[tid + 1] = end;
        sm.kv[tid] = kv;
        sm.first[tid] = head + last_page - static_cast<int>(fresh);
        if (tid == 0)
            sm.cu[0] = tokens;
        if (blockIdx.x == 0 && b < p.batch) {
            p.kv_out[b] = kv + n;
            p.cu_q[b + 1] = end;
        }
        __syncthreads();
        if (t < p.max_tokens && t >= sm.cu[0] && t < sm.cu[kSeqs]) {
            int lo = 0, hi = kSeqs - 1; // the last request that starts at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (sm.cu[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            // (unsigned: lengths that overflow 31 bits find no page)
            const uint32_t pos = static_cast<uint32_t>(sm.kv[lo]) + static_cast<uint32_t>(t - sm.cu[lo]);
            const int page = static_cast<int>(pos >> p.page_shift);
            const int had = static_cast<int>((static_cast<uint32_t>(sm.kv[lo]) + page_mask) >> p.page_shift);
            int id = -1;
            if (page < p.bt_stride && b0 + lo < p.batch) {
                int32_t *entry = p.block_table + static_cast<int64_t>(b0 + lo) * p.bt_stride + page;
                if (page < had) {
                    id = *entry;
                } else {
                    const int at = sm.first[lo] + page - had;
                    if (at >= 0 && at < p.n_free)
                        id = __ldg(p.free_pages + at);
                    if ((pos & page_mask) == 0)
                        *entry = id;
                }
            }
            if (id < 0)
                err |= FL_DEVERR_PAGES;
            p.positions[t] = static_cast<int>(pos);
            if (p.slots)
                p.slots[t] = id < 0 ? -1 : (static_cast<int64_t>(id) << p.page_shift) + (pos & page_mask);
        }
        if (sm.cu[kSeqs] > p.max_tokens)
            err |= unlisted_pages(p, sm, b0, n, kv, static_cast<int>(held), static_cast<int>(held + fresh));
        tokens = sm.cu[kSeqs];
        pages = pages_end;
        __syncthreads(); // the next scan overwrites what was read here
    }
    if (t < p.max_tokens && t >= tokens) {
        p.positions[t] = -1;
        if (p.slots)
            p.slots[t] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.cu_q[0] = 0;
        *p.head_out = head + pages;
        if (p.max_tokens && tokens > p.max_tokens)
            err |= FL_DEVERR_LENGTHS;
    }
    if (err && p.err_user)
        atomicOr(p.err_user, err);
}

} // namespace

cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t stream)
{
    const int grid = p.max_tokens > kTokens ? (p.max_tokens + kTokens - 1) / kTokens : 1;
    kv_plan_kernel<<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

} // namespace fl
