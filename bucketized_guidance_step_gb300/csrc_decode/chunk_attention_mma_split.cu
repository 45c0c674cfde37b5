// Attention of chunks for 16-bit caches: the instances whose weights are sums of two numbers (kernel and launch templates
// in chunk_attention_mma.cuh).
#include "chunk_attention_mma.cuh"

namespace gs_decode {

gs_status launch_chunk_mma_split(int dtype, ChunkParams& p, int blocks, gs_stream stream) {
    return launch_mma<true>(dtype, p, blocks, stream);
}

}  // namespace gs_decode
