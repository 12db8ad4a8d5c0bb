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

#include "kda_attn.cuh"
#include "kda_launch.h"

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
  const int b = lo;
  const Request r = load_request(p, b, true);
  if (t < r.t0 || t >= r.t0 + r.n || r.n * p.G <= kWindowRows) return;
  const int pos = r.L - r.n + (t - r.t0), end = seen_hi(p, pos, r.L), begin = seen_lo(p, pos);

  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = p.scale * __uint_as_float((uint32_t)p.q[t * p.q_stride + (size_t)h * D + lane * E + i] << 16);
    o[i] = 0.f;
  }
  for (int j = begin; j < end; ++j) {
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

// The pieces of one shared item (kda_attn.cuh) into its outputs: with m = max m_i,
//   o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i,   lse = (m + log2 l) ln 2.
// CTA (c, y) takes rows y, y + gridDim.y, .. of the item that CTA c of the main
// kernel began, kJoinWarps warps to a row, each every kJoinWarps-th piece, in order.
constexpr int kJoinWarps = 4;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttentionArgs p, const Pieces s, int rows) {
  constexpr int E = D / 32;
  __shared__ float part[kJoinWarps][D];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x;
  const PieceNote note = s.notes[c];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int row = blockIdx.y; row < note.tokens * p.G; row += gridDim.y) {
    auto at = [&](int i) { return ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * rows + row; };
    float m = -INFINITY;
    for (int i = lane; i < note.pieces; i += 32) m = fmaxf(m, s.ml[at(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int i = lane; i < note.pieces; i += 32) {
      const float2 ml = s.ml[at(i)];
      l += ml.y * exp2_approx(ml.x - ref);
    }
    l = warp_sum(l);
    float o[E] = {};
#pragma unroll 4
    for (int i = warp; i < note.pieces; i += kJoinWarps) {
      const float w = exp2_approx(s.ml[at(i)].x - ref);
      const float* x = s.o + at(i) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = *reinterpret_cast<const float2*>(x + e);
        o[e] = fmaf(w, v.x, o[e]);
        o[e + 1] = fmaf(w, v.y, o[e + 1]);
      }
    }
    __syncthreads();  // the row before has been read
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][lane * E + e] = o[e];
    __syncthreads();
    const int tok = row / p.G;
    const size_t out_row = (size_t)note.row0 + (size_t)tok * p.H + (row - tok * p.G);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int d = threadIdx.x; d < D; d += kJoinWarps * 32) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) sum += part[w][d];
      p.out[out_row * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(sum * inv));
    }
    if (p.lse && threadIdx.x == 0) p.lse[out_row] = (m + log2f(l)) * kLn2;
  }
}

}  // namespace

cudaError_t launch_join_pieces(const AttentionArgs& a, const Pieces& pieces, int rows, int ctas,
                               cudaStream_t stream) {
  const dim3 grid(ctas, rows < 16 ? rows : 16);
  if (a.c.D == 128)
    return launch(join_kernel<128>, grid, dim3(kJoinWarps * 32), 0, stream, true, a, pieces, rows);
  return launch(join_kernel<64>, grid, dim3(kJoinWarps * 32), 0, stream, true, a, pieces, rows);
}

size_t attention_workspace_bytes(int B, int T, int max_tokens, int H, int HKV, int D) {
  if (B < 0 || T < 0 || max_tokens < 0 || H < 1 || HKV < 1 || H % HKV != 0 || (D != 64 && D != 128))
    return 0;
  return (pieces_bytes(window_rows(max_tokens, H / HKV), D) + 255) & ~(size_t)255;
}

cudaError_t launch_paged_attention(const AttentionArgs& a, cudaStream_t stream) {
  const cudaError_t e = launch_window_attention(a, stream);
  if (e != cudaSuccess || (long long)a.max_tokens * a.G <= kWindowRows) return e;
  const long long items = (long long)a.T * a.H;
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
