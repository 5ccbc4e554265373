// rope.cu -- rotary positions of q and k, and the same on the way into a
// paged KV cache (the append of new keys and values).
//
//   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_a sin t + x_b cos t),  t = pos f_i
//
// The angle: f_i / 2 pi is held as a 64-bit fraction of a turn, so pos times
// it, in 64-bit integers, is the angle modulo a turn with no reduction, and all
// that grows with the position is the frequency's own error, a few 2^-53 of it
// (a 32-bit float angle is off by 0.06 rad at position 10^6).  The nearest quarter turn is taken off in integers too;
// the remainder, in [-1/8, 1/8] turn, goes to sincospif.
//
// Bound by HBM: every element is read and written once.  A block takes `tile`
// tokens of one tensor and puts their sines and cosines (one sincos for all
// heads of a token) and row offsets in shared memory.  A thread keeps its
// place within a head -- the two vectors of up to 16 bytes that hold its V
// pairs -- and walks the (token, head) rows with it, so that a unit costs an
// address, two loads, the rotation and two stores (about 90 instructions for
// 8 bf16 pairs; with the place and the tensor worked out for every unit it
// was 290, in 116 registers, and 45 us where this takes 24 for q and k of 8 x
// 2048 tokens of 16 heads of 64).
#include "rope.cuh"

namespace fl {
namespace {

// Occupancy carries the latency (one row in flight a thread, 8 blocks a
// SM): two rows in flight and 4 blocks took 31.8 us, four and 3 42.7.
template <class T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ __align__(16) float2 s_cs[kMaxAngles];
    __shared__ int64_t s_src[kMaxTile], s_dst[kMaxTile];
    rope_tile<T, V, INTER>(p, p.st[blockIdx.y], s_cs, s_src, s_dst);
}

template <class T, int V>
cudaError_t launch_vec(RopeParams &p, bool interleaved, int sm_count, cudaStream_t stream)
{
    const int blocks = rope_shape(p, V, sm_count);
    if (blocks == 0)
        return cudaSuccess;
    const dim3 grid(blocks, p.n_streams);
    if (interleaved)
        rope_kernel<T, V, true><<<grid, kRopeThreads, 0, stream>>>(p);
    else
        rope_kernel<T, V, false><<<grid, kRopeThreads, 0, stream>>>(p);
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
