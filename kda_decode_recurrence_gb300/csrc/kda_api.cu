// kda_api.cu -- the extern "C" boundary of libkda: host-side argument
// validation, then kernel launches on the caller's stream.  No allocation.
#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_internal.h"
#include "kda_paged.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" {

const char* kda_status_string(kda_status status) {
  switch (status) {
    case KDA_OK: return "ok";
    case KDA_ERR_NULL: return "a required pointer is NULL";
    case KDA_ERR_SHAPE: return "a size is out of range or sizes are inconsistent";
    case KDA_ERR_UNSUPPORTED: return "sizes not implemented by this build";
    case KDA_ERR_ENUM: return "unknown gate_mode, state_layout, output_dtype or cache_dtype";
    case KDA_ERR_CUDA: return "a CUDA runtime call failed";
    case KDA_ERR_ALIGN: return "a pointer is not aligned as documented";
    case KDA_ERR_VALUE: return "a scalar argument is not finite or out of range";
    case KDA_ERR_WORKSPACE: return "workspace missing or too small";
  }
  return "unknown status";
}

const char* kda_version(void) { return "kda-gb300 0.1"; }

}  // extern "C"

namespace {

kda_status decode_impl(void* output, const kda_bf16* q, const kda_bf16* k, const kda_bf16* v,
                       const float* raw_gate, const float* beta_logits, const float* a_log,
                       const float* dt_bias, const int32_t* cu_seqlens, float* state_pool,
                       const int32_t* state_indices, int gate_mode, float lower_bound,
                       int state_layout, int output_dtype, int B, int T, int H, int HV, int K,
                       int V, int max_slots, int32_t* dev_status, void* stream,
                       bool prefill = false) {
  if (B < 0 || T < 0 || H < 1 || HV < 1 || K < 1 || V < 1 || max_slots < 1) return KDA_ERR_SHAPE;
  if (HV % H != 0) return KDA_ERR_SHAPE;
  if (gate_mode != KDA_GATE_SOFTPLUS && gate_mode != KDA_GATE_LOWER_BOUND) return KDA_ERR_ENUM;
  if (state_layout != KDA_STATE_K_FIRST && state_layout != KDA_STATE_V_FIRST) return KDA_ERR_ENUM;
  if (output_dtype != KDA_OUTPUT_F32 && output_dtype != KDA_OUTPUT_BF16) return KDA_ERR_ENUM;
  if (gate_mode == KDA_GATE_LOWER_BOUND && !(std::isfinite(lower_bound) && lower_bound <= 0.0f))
    return KDA_ERR_VALUE;
  if (K != kda::kHeadDim || V != kda::kHeadDim) return KDA_ERR_UNSUPPORTED;
  if ((long long)B * HV > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  if (B == 0) return KDA_OK;
  if (!cu_seqlens || !state_pool || !state_indices || !a_log || !dt_bias) return KDA_ERR_NULL;
  if (T > 0 && (!output || !q || !k || !v || !raw_gate || !beta_logits)) return KDA_ERR_NULL;
  if (!aligned(state_pool, 16) || !aligned(dt_bias, 16) || !aligned(cu_seqlens, 4) ||
      !aligned(state_indices, 4) || !aligned(a_log, 4))
    return KDA_ERR_ALIGN;
  const uintptr_t out_align = output_dtype == KDA_OUTPUT_F32 ? 16 : 8;
  if (T > 0 && (!aligned(output, out_align) || !aligned(raw_gate, 16) || !aligned(q, 8) ||
                !aligned(k, 8) || !aligned(v, 8) || !aligned(beta_logits, 4)))
    return KDA_ERR_ALIGN;

  kda::DecodeArgs a;
  a.output = output;
  a.q = q;
  a.k = k;
  a.v = v;
  a.raw_gate = raw_gate;
  a.beta_logits = beta_logits;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.cu_seqlens = cu_seqlens;
  a.state_pool = state_pool;
  a.state_indices = state_indices;
  a.dev_status = dev_status;
  a.gate_mode = gate_mode;
  a.lower_bound = lower_bound;
  a.q_scale = 1.0f / std::sqrt((float)K);
  a.v_first = state_layout == KDA_STATE_V_FIRST;
  a.out_bf16 = output_dtype == KDA_OUTPUT_BF16;
  a.B = B;
  a.T = T;
  a.H = H;
  a.HV = HV;
  a.G = HV / H;
  a.max_slots = max_slots;
  const cudaError_t e = prefill ? kda::launch_kda_prefill(a, static_cast<cudaStream_t>(stream))
                                : kda::launch_kda_decode(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

extern "C" {

kda_status kda_decode(float* output, const kda_bf16* q, const kda_bf16* k, const kda_bf16* v,
                      const float* raw_gate, const float* beta_logits, const float* a_log,
                      const float* dt_bias, const int32_t* cu_seqlens, float* state_pool,
                      const int32_t* state_indices, int gate_mode, float lower_bound, int B,
                      int T, int H, int HV, int K, int V, int max_slots, int32_t* dev_status,
                      void* stream) {
  return decode_impl(output, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens,
                     state_pool, state_indices, gate_mode, lower_bound, KDA_STATE_K_FIRST,
                     KDA_OUTPUT_F32, B, T, H, HV, K, V, max_slots, dev_status, stream);
}

kda_status kda_decode_ex(void* output, const kda_bf16* q, const kda_bf16* k, const kda_bf16* v,
                         const float* raw_gate, const float* beta_logits, const float* a_log,
                         const float* dt_bias, const int32_t* cu_seqlens, float* state_pool,
                         const int32_t* state_indices, int gate_mode, float lower_bound,
                         int state_layout, int output_dtype, int B, int T, int H, int HV, int K,
                         int V, int max_slots, int32_t* dev_status, void* stream) {
  return decode_impl(output, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens,
                     state_pool, state_indices, gate_mode, lower_bound, state_layout,
                     output_dtype, B, T, H, HV, K, V, max_slots, dev_status, stream);
}

kda_status kda_prefill(float* output, const kda_bf16* q, const kda_bf16* k, const kda_bf16* v,
                       const float* raw_gate, const float* beta_logits, const float* a_log,
                       const float* dt_bias, const int32_t* cu_seqlens, float* state_pool,
                       const int32_t* state_indices, int gate_mode, float lower_bound, int B,
                       int T, int H, int HV, int K, int V, int max_slots, int32_t* dev_status,
                       void* stream) {
  // The chunk form needs the decay accumulated over a chunk bounded: the
  // lower-bound gate with lower_bound >= -5 keeps |G| <= 80, so every
  // e^(+-G) factor is a normal fp32 number.  The softplus gate (unbounded
  // decay) and lower bounds below -5 run the token-by-token kernel instead,
  // which computes the same recurrence.
  const bool chunked = !(gate_mode == KDA_GATE_SOFTPLUS ||
                         (gate_mode == KDA_GATE_LOWER_BOUND && std::isfinite(lower_bound) &&
                          lower_bound < -5.0f));
  return decode_impl(output, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens,
                     state_pool, state_indices, gate_mode, lower_bound, KDA_STATE_K_FIRST,
                     KDA_OUTPUT_F32, B, T, H, HV, K, V, max_slots, dev_status, stream, chunked);
}

size_t kda_block_tkg_workspace_size(int B, int n, int Hd, int nh, int K, int V, int Kc) {
  return kda::block_workspace_bytes(B, n, Hd, nh, K, V, Kc);
}

kda_status kda_block_tkg(float* out, const float* hidden, const float* gamma_in,
                         const kda_bf16* W_in, const kda_bf16* W_fb, const kda_bf16* W_gb,
                         const kda_bf16* conv_w, const float* A_log, const float* dt_bias,
                         const float* gamma_o, const kda_bf16* W_o, float* S, float* conv_state,
                         float scale, float lower_bound, float rms_norm_eps, float l2_eps, int B,
                         int n, int Hd, int nh, int K, int V, int Kc, void* workspace,
                         size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (B < 0 || n < 1 || Hd < 1 || nh < 1 || K < 1 || V < 1 || Kc < 1) return KDA_ERR_SHAPE;
  if (!(std::isfinite(scale) && std::isfinite(lower_bound) && lower_bound <= 0.0f &&
        std::isfinite(rms_norm_eps) && rms_norm_eps >= 0.0f && std::isfinite(l2_eps) &&
        l2_eps >= 0.0f))
    return KDA_ERR_VALUE;
  if (K != kda::kHeadDim || V != kda::kHeadDim || Kc < 2 ||
      Kc > 4 || Hd % 128 != 0)
    return KDA_ERR_UNSUPPORTED;
  if (B == 0) return KDA_OK;
  if (!out || !hidden || !gamma_in || !W_in || !W_fb || !W_gb || !conv_w || !A_log ||
      !dt_bias || !gamma_o || !W_o || !S || !conv_state)
    return KDA_ERR_NULL;
  const void* ptrs[] = {out, hidden, gamma_in, W_in, W_fb, W_gb, conv_w, A_log,
                        dt_bias, gamma_o, W_o, S, conv_state};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return KDA_ERR_ALIGN;
  const size_t need = kda::block_workspace_bytes(B, n, Hd, nh, K, V, Kc);
  if (need == 0) return KDA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KDA_ERR_ALIGN;

  kda::BlockArgs a;
  a.out = out;
  a.hidden = hidden;
  a.gamma_in = gamma_in;
  a.W_in = W_in;
  a.W_fb = W_fb;
  a.W_gb = W_gb;
  a.conv_w = conv_w;
  a.A_log = A_log;
  a.dt_bias = dt_bias;
  a.gamma_o = gamma_o;
  a.W_o = W_o;
  a.S = S;
  a.conv_state = conv_state;
  a.scale = scale;
  a.lower_bound = lower_bound;
  a.rms_norm_eps = rms_norm_eps;
  a.l2_eps = l2_eps;
  a.B = B;
  a.n = n;
  a.Hd = Hd;
  a.nh = nh;
  a.K = K;
  a.V = V;
  a.Kc = Kc;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.dev_status = dev_status;
  if (kda::launch_kda_block(a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return KDA_ERR_CUDA;
  return KDA_OK;
}

}  // extern "C"

namespace {

// What every call on a paged cache checks first; fills `c` when it returns KDA_OK.
kda_status check_cache(kda::PagedCache& c, const void* k, const void* v, const float* k_scale,
                       const float* v_scale, const int32_t* page_table, int cache_dtype, int B,
                       int T, int HKV, int D, int page_size, int num_pages, int max_pages) {
  if (B < 0 || T < 0 || HKV < 1 || D < 1 || page_size < 1 || num_pages < 1 || max_pages < 1)
    return KDA_ERR_SHAPE;
  if (cache_dtype != KDA_CACHE_BF16 && cache_dtype != KDA_CACHE_E4M3) return KDA_ERR_ENUM;
  if ((D != 64 && D != 128) ||
      (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128))
    return KDA_ERR_UNSUPPORTED;
  // Positions are 32-bit, and so are row numbers of the cache (a copy's coordinate).
  if (HKV > 4096 || (long long)max_pages * page_size > 0x40000000LL ||
      (long long)num_pages * HKV > (0x7fffffffLL - 128) / page_size || (long long)T * HKV > 0x3fffffffLL)
    return KDA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return KDA_OK;
  const bool e4m3 = cache_dtype == KDA_CACHE_E4M3;
  if (!k || !v || !page_table || (e4m3 && (!k_scale || !v_scale))) return KDA_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(page_table, 4) || !aligned(k_scale, 16) ||
      !aligned(v_scale, 16))
    return KDA_ERR_ALIGN;
  c.k = const_cast<void*>(k);
  c.v = const_cast<void*>(v);
  c.k_scale = e4m3 ? const_cast<float*>(k_scale) : nullptr;
  c.v_scale = e4m3 ? const_cast<float*>(v_scale) : nullptr;
  c.page_table = page_table;
  c.e4m3 = e4m3;
  c.HKV = HKV;
  c.D = D;
  c.page_size = page_size;
  c.num_pages = num_pages;
  c.max_pages = max_pages;
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_cache_append(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                            const kda_bf16* k, const kda_bf16* v, const int32_t* cu_seqlens,
                            const int32_t* seq_lens, const int32_t* page_table, int cache_dtype,
                            int B, int T, int HKV, int D, int page_size, int num_pages,
                            int max_pages, long long k_stride, long long v_stride,
                            int32_t* dev_status, void* stream) {
  kda::CacheRowsArgs a = {};
  const kda_status st = check_cache(a.c, k_cache, v_cache, k_scale, v_scale, page_table,
                                    cache_dtype, B, T, HKV, D, page_size, num_pages, max_pages);
  if (st != KDA_OK) return st;
  const long long row = (long long)HKV * D;
  if (k_stride < row || v_stride < row) return KDA_ERR_SHAPE;
  if (B == 0 || T == 0) return KDA_OK;
  if (!k || !v || !cu_seqlens || !seq_lens) return KDA_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 != 0 || v_stride % 8 != 0 ||
      !aligned(cu_seqlens, 4) || !aligned(seq_lens, 4))
    return KDA_ERR_ALIGN;
  a.k_rows = const_cast<kda_bf16*>(k);
  a.v_rows = const_cast<kda_bf16*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu = cu_seqlens;
  a.at = seq_lens;
  a.B = B;
  a.T = T;
  a.dev_status = dev_status;
  return kda::launch_cache_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_cache_read(kda_bf16* k_rows, kda_bf16* v_rows, const void* k_cache,
                          const void* v_cache, const float* k_scale, const float* v_scale,
                          const int32_t* cu_rows, const int32_t* starts, const int32_t* page_table,
                          int cache_dtype, int B, int T, int HKV, int D, int page_size,
                          int num_pages, int max_pages, int32_t* dev_status, void* stream) {
  kda::CacheRowsArgs a = {};
  const kda_status st = check_cache(a.c, k_cache, v_cache, k_scale, v_scale, page_table,
                                    cache_dtype, B, T, HKV, D, page_size, num_pages, max_pages);
  if (st != KDA_OK || B == 0 || T == 0) return st;
  if (!k_rows || !v_rows || !cu_rows) return KDA_ERR_NULL;
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(cu_rows, 4) || !aligned(starts, 4))
    return KDA_ERR_ALIGN;
  a.k_rows = k_rows;
  a.v_rows = v_rows;
  a.k_stride = a.v_stride = (long long)HKV * D;
  a.cu = cu_rows;
  a.at = starts;
  a.B = B;
  a.T = T;
  a.dev_status = dev_status;
  return kda::launch_cache_read(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_paged_attention_workspace_size(int B, int T, int max_tokens, int H, int HKV, int D) {
  return kda::attention_workspace_bytes(B, T, max_tokens, H, HKV, D);
}

kda_status kda_paged_attention(kda_bf16* out, float* lse, const kda_bf16* q, const void* k_cache,
                               const void* v_cache, const float* k_scale, const float* v_scale,
                               const int32_t* cu_seqlens, const int32_t* seq_lens,
                               const int32_t* page_table, float scale, int causal, int window,
                               int cache_dtype, int B, int T, int max_tokens, int H, int HKV,
                               int D, int page_size, int num_pages, int max_pages,
                               long long q_stride, void* workspace, size_t workspace_bytes,
                               int32_t* dev_status, void* stream) {
  kda::AttentionArgs a = {};
  const kda_status st = check_cache(a.c, k_cache, v_cache, k_scale, v_scale, page_table,
                                    cache_dtype, B, T, HKV, D, page_size, num_pages, max_pages);
  if (st != KDA_OK) return st;
  if (H < 1 || H % HKV != 0 || max_tokens < 0 || q_stride < (long long)H * D) return KDA_ERR_SHAPE;
  if (H / HKV > 128 || (long long)T * H > 0x3fffffffLL) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || window < 0 || (causal != 0 && causal != 1)) return KDA_ERR_VALUE;
  if (B == 0 || T == 0) return KDA_OK;
  if (!out || !q || !cu_seqlens || !seq_lens) return KDA_ERR_NULL;
  if (!aligned(out, 16) || !aligned(q, 16) || q_stride % 8 != 0 || !aligned(lse, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(seq_lens, 4))
    return KDA_ERR_ALIGN;
  if (!workspace || workspace_bytes < kda::attention_workspace_bytes(B, T, max_tokens, H, HKV, D))
    return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KDA_ERR_ALIGN;
  a.out = out;
  a.lse = lse;
  a.q = q;
  a.q_stride = q_stride;
  a.cu = cu_seqlens;
  a.lens = seq_lens;
  a.scale = scale;
  a.causal = causal;
  a.window = window < 0x40000000 ? window : 0x40000000;  // longer than any sequence
  a.B = B;
  a.T = T;
  a.max_tokens = max_tokens;
  a.H = H;
  a.G = H / HKV;
  a.workspace = workspace;
  a.dev_status = dev_status;
  return kda::launch_paged_attention(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_verify_draft(int32_t* tokens, int32_t* accepted, const float* target_probs,
                            const float* draft_probs, const int32_t* draft_tokens,
                            const float* accept_u, const float* sample_u, const int32_t* cu_drafts,
                            int B, int N, int V, long long target_stride, long long draft_stride,
                            int32_t* dev_status, void* stream) {
  if (B < 0 || N < 0 || V < 1 || target_stride < V || (draft_probs && draft_stride < V))
    return KDA_ERR_SHAPE;
  if (B > 0x7fffffff / 8 || V > 0x7fffffff - 4096 || (long long)N + B > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  if (B == 0) return KDA_OK;
  if (!tokens || !accepted || !target_probs || !sample_u || !cu_drafts ||
      (N > 0 && (!draft_tokens || !accept_u)))
    return KDA_ERR_NULL;
  const void* ptrs[] = {tokens, accepted, target_probs, draft_probs, draft_tokens,
                        accept_u, sample_u, cu_drafts};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return KDA_ERR_ALIGN;
  kda::VerifyArgs a = {};
  a.tokens = tokens;
  a.accepted = accepted;
  a.target = target_probs;
  a.draft = draft_probs;
  a.draft_tokens = draft_tokens;
  a.accept_u = accept_u;
  a.sample_u = sample_u;
  a.cu = cu_drafts;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.B = B;
  a.N = N;
  a.V = V;
  a.dev_status = dev_status;
  return kda::launch_verify_draft(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
