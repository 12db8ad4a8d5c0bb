// kda_latent.h -- argument bundles of the latent-cache and latent-attention calls,
// passed from the C ABI layer to the launchers (no ownership).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// A latent row: kLatent entries that are keys and values at once, then kRope key entries
// that tell the position.
constexpr int kLatent = 512, kRope = 64, kLatentRow = kLatent + kRope;
// An expanded head: kExpanded key entries of its own beside the shared kRope, kExpanded values.
constexpr int kExpanded = 128;

struct LatentCache {
  kda_bf16* rows;  // [num_pages, page_size, kLatentRow]
  const int32_t* page_table;
  int page_size, num_pages, max_pages;
};

struct LatentAppendArgs {
  LatentCache c;
  const kda_bf16* rows;  // [T, kLatentRow], `stride` elements between tokens
  long long stride;
  const float* gamma;    // [kLatent], or null: rows as they are
  float eps;
  const int32_t* cu;
  const int32_t* lens;
  int B, T;
  int32_t* dev_status;
};

cudaError_t launch_latent_append(const LatentAppendArgs& args, cudaStream_t stream);

struct LatentArgs {
  LatentCache c;
  kda_bf16* out;  // [T, H, kLatent]
  float* lse;     // nullable
  const kda_bf16* q;
  long long q_stride;
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* mask;  // [T, mask_words] bits of the new tokens that a token sees, or null
  int mask_words;
  float scale;
  int causal;
  int B, T, H;
  void* workspace;
  int32_t* dev_status;
};

size_t latent_workspace_bytes(int B, int T, int H);
cudaError_t launch_latent_attention(const LatentArgs& args, cudaStream_t stream);

struct ExpandedArgs {
  kda_bf16* out;  // [Tq, H, kExpanded]
  float* lse;     // nullable
  const kda_bf16* q;
  const kda_bf16* kv;    // [Tk, H, 2 kExpanded]
  const kda_bf16* k_pe;  // [Tk, kRope]
  long long q_stride, kv_stride, pe_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  float scale;
  int causal;
  int B, Tq, Tk, H;
  void* workspace;
  int32_t* dev_status;
};

size_t expanded_workspace_bytes(int B, int Tq, int H);
cudaError_t launch_latent_expanded(const ExpandedArgs& args, cudaStream_t stream);

}  // namespace kda
