// kda_attention.cu -- attention of new tokens over a paged cache.
//
//   token i of request b sits at position p = lens[b] - n_b + i;
//   x_j = scale q . k_j over the positions j it sees:
//     j <= p (causal), j > p - window (window > 0), 0 <= j < lens[b]
//   m = max x_j, l = sum e^(x_j - m), o = sum e^(x_j - m) v_j / l,
//   lse = m + ln l; a token that sees nothing gets o = 0, lse = -inf.
//
// One warp per (token, query head) walks the visible positions with the
// running maximum and sum; lanes split the head dimension.
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_paged.h"

namespace kda {
namespace {

constexpr int kWarps = 8;

template <int D, bool kE4m3>
__device__ __forceinline__ void load_row(const void* cache, const float* scales, size_t row, int lane,
                                         float (&x)[D / 32]) {
  constexpr int E = D / 32;
  if (kE4m3) {
    const uint8_t* src = static_cast<const uint8_t*>(cache) + row * D + lane * E;
    const float s = scales[row];
#pragma unroll
    for (int i = 0; i < E; ++i)
      x[i] = s * __half2float(__half(__nv_cvt_fp8_to_halfraw(src[i], __NV_E4M3)));
  } else {
    const kda_bf16* src = static_cast<const kda_bf16*>(cache) + row * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __uint_as_float((uint32_t)src[i] << 16);
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttentionArgs p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (long long)p.T * p.H) return;
  const int t = (int)(item / p.H), h = (int)(item % p.H);
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  const int b = lo, t0 = p.cu[b], t1 = p.cu[b + 1];
  const long long L = p.lens[b];
  if (t < t0 || t >= t1 || t0 < 0 || t1 > p.T || t1 - t0 > p.max_tokens || L < 0 ||
      L > (long long)p.c.max_pages * p.c.page_size) {
    if (lane == 0) raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
    return;
  }
  const long long pos = L - (t1 - t);
  const long long end = p.causal ? min(L, pos + 1) : (pos < 0 ? 0 : L);
  const long long begin = p.window > 0 ? max(0ll, pos - p.window + 1) : 0;

  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = p.scale * __uint_as_float((uint32_t)p.q[t * p.q_stride + (size_t)h * D + lane * E + i] << 16);
    o[i] = 0.f;
  }
  for (long long j = begin; j < end; ++j) {
    const int page = p.c.page_table[(size_t)b * p.c.max_pages + j / p.c.page_size];
    float k[E] = {}, v[E] = {};
    if (page < 0 || page >= p.c.num_pages) {
      if (lane == 0) raise_status(p.dev_status, KDA_DEV_BAD_PAGE);
    } else {
      const size_t row = ((size_t)page * p.c.HKV + h / p.G) * p.c.page_size + j % p.c.page_size;
      load_row<D, kE4m3>(p.c.k, p.c.k_scale, row, lane, k);
      load_row<D, kE4m3>(p.c.v, p.c.v_scale, row, lane, v);
    }
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) x = fmaf(q[i], k[i], x);
    x = warp_sum(x);
    const float top = fmaxf(m, x);
    const float ref = fmaxf(top, -1e30f);  // finite: a score of -inf weighs 0
    const float keep = expf(m - ref), w = expf(x - ref);
    l = l * keep + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * keep + w * v[i];
    m = top;
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int i = 0; i < E; ++i)
    p.out[((size_t)t * p.H + h) * D + lane * E + i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
  if (p.lse && lane == 0) p.lse[(size_t)t * p.H + h] = m + logf(l);  // nothing seen: -inf - inf
}

}  // namespace

size_t attention_workspace_bytes(int B, int T, int max_tokens, int H, int HKV, int D) {
  if (B < 0 || T < 0 || max_tokens < 0 || H < 1 || HKV < 1 || H % HKV != 0 || (D != 64 && D != 128))
    return 0;
  return 256;
}

cudaError_t launch_paged_attention(const AttentionArgs& a, cudaStream_t stream) {
  const long long items = (long long)a.T * a.H;
  if (items == 0) return cudaSuccess;
  const unsigned grid = (unsigned)((items + kWarps - 1) / kWarps);
  if (a.c.D == 128) {
    if (a.c.e4m3) attention_kernel<128, true><<<grid, kWarps * 32, 0, stream>>>(a);
    else attention_kernel<128, false><<<grid, kWarps * 32, 0, stream>>>(a);
  } else {
    if (a.c.e4m3) attention_kernel<64, true><<<grid, kWarps * 32, 0, stream>>>(a);
    else attention_kernel<64, false><<<grid, kWarps * 32, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace kda
