// kda_attn_tree.cu -- attention of drafted trees over a paged K/V cache, by the size of a head.
//
// Heads of 128 have a kernel of pairs of CTAs (kda_attn_tree_pairs.cu).  Heads of 64 take the chunk kernel
// with a mask of the new tokens that each of them sees: V would have 32 columns per CTA of a pair, half of
// a swizzled row.  (32 trees of 8-60 nodes over 1000-8000, 32 / 8 heads of 64, bf16: 114 us; 16 of 4-32 over 500-12000,
// 96 / 8, e4m3: 219 us; one of 13 over 517: 16 us.  DRAM 27 and 8 %, tensor cores 24 and 15 %, issue 36 and 46 %: a row
// tile's chain bounds it, which takes as long as with heads of 128 for half of the products.)
//
// Trees of a few nodes take these too.  Their rows (nodes x query heads per key head) are mostly more
// than the 16 up to which the window kernel wins over bf16, and everything before the tree is seen by
// every row, so that only the last key tiles differ from a chunk's.
#include "kda_attn_chunk.cuh"

namespace kda {

size_t tree_workspace_bytes(int B, int T, int max_tokens, int H, int HKV, int D) {
  if (B < 0 || T < 0 || max_tokens < 0 || H < 1 || HKV < 1 || H % HKV != 0 || (D != 64 && D != 128)) return 0;
  return D == 128 ? tree_pairs_bytes() : (pieces_bytes(kChunkCtas, kChunkRows, D) + 255) & ~(size_t)255;
}

cudaError_t launch_tree_attention(const AttentionArgs& in, cudaStream_t stream) {
  AttentionArgs a = in;
  a.window_rows = 0;
  if (a.c.D == 128) return launch_tree_pairs(a, stream);
  return a.c.e4m3 ? by_pair<true, 64, true>(a, stream) : by_pair<true, 64, false>(a, stream);
}

}  // namespace kda
