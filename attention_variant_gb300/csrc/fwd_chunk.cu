// fwd_chunk.cu -- attention of ragged chunks of new tokens over a cache in
// bf16: the kernels of chunk_blocks.cuh and chunk_few.cuh.
#include "chunk_blocks.cuh"

namespace fl {

cudaError_t launch_chunk(const ChunkMaps &maps, const ChunkParams &params, cudaStream_t stream)
{
    ChunkParams p = params;
    if (p.head_dim == 64)
        return p.score_mod == MOD_SOFTCAP ? launch_mod<MOD_SOFTCAP, 64, false>(maps, p, stream)
                                          : launch_mod<MOD_NONE, 64, false>(maps, p, stream);
    return p.score_mod == MOD_SOFTCAP ? launch_mod<MOD_SOFTCAP, 128, false>(maps, p, stream)
                                      : launch_mod<MOD_NONE, 128, false>(maps, p, stream);
}

} // namespace fl
