// kda_attn_chunk.cu -- the chunk kernel for the requests of kda_paged_attention that the window
// kernel does not take.
#include "kda_attn_chunk.cuh"

namespace kda {

cudaError_t launch_chunk_attention(const AttentionArgs& a, cudaStream_t stream) { return by_type<false>(a, stream); }

}  // namespace kda
