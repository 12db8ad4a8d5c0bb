// kda_paged.h -- argument bundles of the paged-cache and draft-verification
// calls, passed from the C ABI layer to the launchers (no ownership).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// A K/V cache in pages: [num_pages, HKV, page_size, D] bf16 or e4m3 codes, the
// latter with fp32 scales [num_pages, HKV, page_size]; page_table [B, max_pages].
struct PagedCache {
  void* k;
  void* v;
  float* k_scale;  // null for bf16
  float* v_scale;
  const int32_t* page_table;
  int e4m3;
  int HKV, D, page_size, num_pages, max_pages;
};

struct CacheRowsArgs {
  PagedCache c;
  kda_bf16* k_rows;  // append reads them, read writes them
  kda_bf16* v_rows;
  long long k_stride, v_stride;  // elements between two tokens' rows
  const int32_t* cu;             // [B + 1] packed rows per request
  const int32_t* at;             // append: cached length with the new rows; read: first position
  int B, T;
  int32_t* dev_status;
};

cudaError_t launch_cache_append(const CacheRowsArgs& args, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheRowsArgs& args, cudaStream_t stream);

struct AttentionArgs {
  PagedCache c;
  kda_bf16* out;
  float* lse;  // nullable
  const kda_bf16* q;
  long long q_stride;
  const int32_t* cu;
  const int32_t* lens;
  float scale;
  int causal, window;
  int B, T, max_tokens, H, G;
  int window_rows;  // requests of at most so many rows are the window kernel's
  const int32_t* tree;  // [T, tree_words] bits of the new tokens that a token sees (trees only)
  int tree_words;       // 32 tree_words >= max_tokens
  void* workspace;
  int32_t* dev_status;
};

size_t attention_workspace_bytes(int B, int T, int max_tokens, int H, int HKV, int D);
cudaError_t launch_paged_attention(const AttentionArgs& args, cudaStream_t stream);

size_t tree_workspace_bytes(int B, int T, int max_tokens, int H, int HKV, int D);
cudaError_t launch_tree_attention(const AttentionArgs& args, cudaStream_t stream);
size_t tree_pairs_bytes();
cudaError_t launch_tree_pairs(const AttentionArgs& args, cudaStream_t stream);  // heads of 128

struct VerifyArgs {
  int32_t* tokens;
  int32_t* accepted;
  const float* target;
  const float* draft;  // null: each draft token was proposed with certainty
  const int32_t* draft_tokens;
  const float* accept_u;
  const float* sample_u;
  const int32_t* cu;
  long long target_stride, draft_stride;
  int B, N, V;
  int32_t* dev_status;
};

cudaError_t launch_verify_draft(const VerifyArgs& args, cudaStream_t stream);

}  // namespace kda
