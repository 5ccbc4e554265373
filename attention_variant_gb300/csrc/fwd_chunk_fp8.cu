// fwd_chunk_fp8.cu -- attention of ragged chunks of new tokens over a cache in
// 8 bits: the kernels of chunk_blocks.cuh and chunk_few.cuh (mathematics, bounds and
// figures there).  A unit of its own, compiled beside fwd_chunk.cu.
#include "chunk_blocks.cuh"

namespace fl {

cudaError_t launch_chunk_fp8(const ChunkMaps &maps, const ChunkParams &params, cudaStream_t stream)
{
    ChunkParams p = params;
    if (p.head_dim == 64)
        return p.score_mod == MOD_SOFTCAP ? launch_mod<MOD_SOFTCAP, 64, true>(maps, p, stream)
                                          : launch_mod<MOD_NONE, 64, true>(maps, p, stream);
    return p.score_mod == MOD_SOFTCAP ? launch_mod<MOD_SOFTCAP, 128, true>(maps, p, stream)
                                      : launch_mod<MOD_NONE, 128, true>(maps, p, stream);
}

} // namespace fl
