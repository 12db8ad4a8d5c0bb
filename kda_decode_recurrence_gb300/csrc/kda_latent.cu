// kda_latent.cu -- new tokens' latent rows into a paged latent cache (kda_latent_append).
//
//   row = (c, p), 512 + 64 entries;  with gamma:  c' = bf16(c (mean c^2 + eps)^-1/2 gamma)
//
// 2304 bytes are moved per token on some 1600 operations: HBM bounds it.  A warp takes a token's
// 72 chunks of 16 bytes (two to each lane, and one of p to the first eight), kUnroll tokens in
// flight, the places of its tokens looked up by its lanes at once.
//
// 9 prompts of 1000-8191 tokens: 16.5 us, 4.9 TB/s (a copy: 6.7); the sum over a warp and a token's place are
// waits that loads of other tokens cover (issue 49 %, DRAM 32 % with cold caches).  Tokens per warp x tokens
// in flight: 2 x 2 17.7 us, 4 x 2 16.5, 8 x 2 16.8, 16 x 4 17.9, 8 x 4 19.1.
#include "kda_common.cuh"
#include "kda_latent.h"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 2;

__device__ __forceinline__ bool good_request(const LatentAppendArgs& p, int t0, int t1, int len) {
  return t0 >= 0 && t1 >= t0 && t1 <= p.T && len >= 0 && len <= (long long)p.c.max_pages * p.c.page_size;
}

// Row of the cache of packed token t; -1: it has no place.
__device__ __forceinline__ int find_row(const LatentAppendArgs& p, int t) {
  const int b = find_request(p.cu, p.B, t);
  const int t0 = fresh(p.cu + b), t1 = fresh(p.cu + b + 1), len = fresh(p.lens + b);
  if (t < t0 || t >= t1 || !good_request(p, t0, t1, len)) return -1;
  const int pos = len - (t1 - t);
  if (pos < 0) return -1;  // padding before the sequence's first position
  const int page = fresh(p.c.page_table + (size_t)b * p.c.max_pages + pos / p.c.page_size);
  if (page < 0 || page >= p.c.num_pages) {
    raise_status(p.dev_status, KDA_DEV_BAD_PAGE);
    return -1;
  }
  return page * p.c.page_size + pos % p.c.page_size;
}

// kTiny: eps is below 2^-90, so that a small row's squares count.  (An instance of its own: with the small rows'
// factor in every call the prompts take 17.3 us in place of 16.5.)
template <bool kNorm, bool kTiny>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs p, int tokens) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) {  // one more CTA looks at every request
    bool bad = threadIdx.x == 0 && (fresh(p.cu) != 0 || fresh(p.cu + p.B) != p.T);
    for (int b = threadIdx.x; b < p.B; b += kThreads)
      bad |= !good_request(p, fresh(p.cu + b), fresh(p.cu + b + 1), fresh(p.lens + b));
    if (bad) raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
    return;
  }
  const int lane = threadIdx.x & 31;
  const long long first = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * tokens;
  if (first >= p.T) return;
  const int t0 = (int)first, count = min(tokens, p.T - t0);
  const int place = lane < count ? find_row(p, t0 + lane) : -1;
  float g[16];
  if constexpr (kNorm) {
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p.gamma + (e >> 3) * 256 + lane * 8 + (e & 7)));
      g[e] = x.x;
      g[e + 1] = x.y;
      g[e + 2] = x.z;
      g[e + 3] = x.w;
    }
  }
  for (int i0 = 0; i0 < count; i0 += kUnroll) {
    uint4 x[kUnroll][3];
    int row[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u;
      row[u] = i < count ? __shfl_sync(0xffffffffu, place, i & 31) : -1;
      if (row[u] < 0) continue;
      const uint4* src = reinterpret_cast<const uint4*>(p.rows + (size_t)(t0 + i) * p.stride);
      x[u][0] = src[lane];
      x[u][1] = src[32 + lane];
      if (lane < 8) x[u][2] = src[64 + lane];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (row[u] < 0) continue;
      if constexpr (kNorm) {
        float c[16], sum = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t w[4] = {x[u][k].x, x[u][k].y, x[u][k].z, x[u][k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[8 * k + 2 * e] = bf16_lo(w[e]);
            c[8 * k + 2 * e + 1] = bf16_hi(w[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) sum = fmaf(c[e], c[e], sum);
        sum = warp_sum(sum);
        // Squares past fp32, or below it where eps is too: the row is scaled by a power of two first.  (1 / rms of a
        // small row may pass fp32, since the smallest bf16 is 2^-133: 2^12 of it goes to the entries.)
        float f = 1.f;
        if (sum == INFINITY) f = 0x1p-72f;
        else if (kTiny && sum < 0x1p-90f) f = 0x1p100f;
        if (f != 1.f) {
          sum = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) sum = fmaf(c[e] * f, c[e] * f, sum);
          sum = warp_sum(sum);
        }
        const float inv = __frsqrt_rn(fmaf(sum, 1.f / kLatent, p.eps * f * f)) * (kTiny ? fminf(f, 0x1p88f) : f);
        if (kTiny && f > 1.f) {
#pragma unroll
          for (int e = 0; e < 16; ++e) c[e] *= 0x1p12f;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = 8 * k + 2 * e;
            const __nv_bfloat162 y = __floats2bfloat162_rn(c[at] * inv * g[at], c[at + 1] * inv * g[at + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&y);
          }
          x[u][k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      uint4* to = reinterpret_cast<uint4*>(p.c.rows + (size_t)row[u] * kLatentRow);
      to[lane] = x[u][0];
      to[32 + lane] = x[u][1];
      if (lane < 8) to[64 + lane] = x[u][2];
    }
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, cudaStream_t stream) {
  // Four tokens to a warp where there are enough for all SMs, else one.
  const int tokens = a.T >= 152 * 4 * kWarps * 2 ? 4 : 1;
  const long long per_cta = (long long)kWarps * tokens;
  const dim3 grid((unsigned)((a.T + per_cta - 1) / per_cta + 1));
  auto* kernel = !a.gamma ? latent_append_kernel<false, false>
                          : a.eps < 0x1p-90f ? latent_append_kernel<true, true> : latent_append_kernel<true, false>;
  return launch(kernel, grid, dim3(kThreads), 0, stream, true, a, tokens);
}

}  // namespace kda
