// kda_attn_chunk.cu -- the chunk kernel for the requests of kda_paged_attention that the window
// kernel does not take.
#include "kda_attn_chunk.cuh"

namespace kda {

cudaError_t launch_chunk_attention(const AttentionArgs& a, cudaStream_t stream) {
  if (a.c.D == 128) return a.c.e4m3 ? by_pair<false, 128, true>(a, stream) : by_pair<false, 128, false>(a, stream);
  return a.c.e4m3 ? by_pair<false, 64, true>(a, stream) : by_pair<false, 64, false>(a, stream);
}

}  // namespace kda
