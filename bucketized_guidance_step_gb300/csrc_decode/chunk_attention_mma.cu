// Attention of chunks for 16-bit caches: the instances whose weights are rounded to the cache's type (kernel and launch
// templates in chunk_attention_mma.cuh).
#include "chunk_attention_mma.cuh"

namespace gs_decode {

ChunkShape chunk_mma_shape(int dim) { return {dim > 128 ? 128 : 256, sm_count()}; }

gs_status launch_chunk_mma(int dtype, ChunkParams& p, int blocks, gs_stream stream) {
    return launch_mma<false>(dtype, p, blocks, stream);
}

}  // namespace gs_decode
