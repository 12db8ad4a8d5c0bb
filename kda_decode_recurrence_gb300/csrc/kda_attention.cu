// kda_attention.cu -- attention of new tokens over a paged cache.
//
//   token i of request b sits at position p = lens[b] - n_b + i;
//   x_j = scale q . k_j over the positions j it sees:
//     j <= p (causal), j > p - window (window > 0), 0 <= j < lens[b]
//   m = max x_j, l = sum e^(x_j - m), o = sum e^(x_j - m) v_j / l,
//   lse = m + ln l; a token that sees nothing gets o = 0, lse = -inf.
//
// Requests with few rows (tokens x query heads per key head: window_limit) go to the
// window kernel (kda_attn_window.cu: HBM-bound), the others to the chunk kernel
// (kda_attn_chunk.cu: tensor-bound); a call that may have both launches both.  Both
// leave the items that several CTAs share in pieces for the join kernel below.
#include "kda_attn.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

// The pieces of one shared item (kda_attn.cuh) into its outputs: with m = max m_i,
//   o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i,   lse = (m + log2 l) ln 2.
// CTA (c, y) takes rows of the item that CTA c of the main kernel began: a warp to a
// row, or all four to a row (each every fourth piece, in order) where an item is in
// many pieces.  Latency bounds it: dependent reads of what the main kernel has just
// written.
constexpr int kJoinWarps = 4;
constexpr int kManyPieces = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttentionArgs p, const Pieces s, int rows) {
  constexpr int E = D / 32;
  __shared__ float part[kJoinWarps][D];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x;
  const PieceNote note = s.notes[c];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool many = note.pieces > kManyPieces;
  const int row0 = many ? blockIdx.y : blockIdx.y * kJoinWarps + warp;
  const int row_step = many ? gridDim.y : gridDim.y * kJoinWarps;
  const int first = many ? warp : 0, step = many ? kJoinWarps : 1;
  for (int row = row0; row < note.tokens * p.G; row += row_step) {
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
    for (int i = first; i < note.pieces; i += step) {
      const float w = exp2_approx(s.ml[at(i)].x - ref);
      const float* x = s.o + at(i) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = *reinterpret_cast<const float2*>(x + e);
        o[e] = fmaf(w, v.x, o[e]);
        o[e + 1] = fmaf(w, v.y, o[e + 1]);
      }
    }
    const int tok = row / p.G;
    const size_t out_row = (size_t)note.row0 + (size_t)tok * p.H + (row - tok * p.G);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (many) {
      __syncthreads();  // the row before has been read
#pragma unroll
      for (int e = 0; e < E; ++e) part[warp][lane * E + e] = o[e];
      __syncthreads();
      if (warp > 0) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) o[e] += part[w][lane * E + e];
      }
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(p.out + out_row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) to[e / 2] = pack_bf16(o[e] * inv, o[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[out_row] = (m + log2f(l)) * kLn2;
  }
}

}  // namespace

cudaError_t launch_join_pieces(const AttentionArgs& a, const Pieces& pieces, int rows, int ctas,
                               cudaStream_t stream) {
  const dim3 grid(ctas, rows <= 64 ? rows / 4 : 32);
  if (a.c.D == 128)
    return launch(join_kernel<128>, grid, dim3(kJoinWarps * 32), 0, stream, true, a, pieces, rows);
  return launch(join_kernel<64>, grid, dim3(kJoinWarps * 32), 0, stream, true, a, pieces, rows);
}

// Whether a call may launch the chunk kernel; others need no room for its pieces.
static bool may_chunk(int max_tokens, int G) { return (long long)max_tokens * G > 16; }

size_t attention_workspace_bytes(int B, int T, int max_tokens, int H, int HKV, int D) {
  if (B < 0 || T < 0 || max_tokens < 0 || H < 1 || HKV < 1 || H % HKV != 0 || (D != 64 && D != 128))
    return 0;
  const int G = H / HKV;
  size_t need = pieces_bytes(kWindowCtas, window_rows(max_tokens, G), D);
  if (may_chunk(max_tokens, G)) {
    const size_t chunk = pieces_bytes(kChunkCtas, kChunkRows, D);
    if (chunk > need) need = chunk;  // the kernels take their turns
  }
  return (need + 255) & ~(size_t)255;
}

// Rows up to which a request is the window kernel's (none: 0).  Measured with 32 requests
// over 200 .. 6000 positions, 8 key heads of 128, window kernel against chunk kernel: e4m3 (from
// a cold L2) 20 rows 110 us against 138, 32 rows 114 against 140, 1 to 8 tokens of 4 heads 106
// against 139; with a warm one 64 rows 206 against 158; bf16 20 rows 99 against 85, 32 rows 118
// against 87.  bf16 windows that differ, the chunk kernel for all against the window kernel
// for the short ones: 1 to 8 tokens of 4 heads 86 us against 95, 1 to 16 85 against 112 (128
// requests of up to 16000 positions 664 against 689), 1 to 8 of 8 heads of 64 55 against 73.
// Longer chunks may come with many single tokens, which are HBM's.
int window_limit(const AttentionArgs& a) {
  if (a.c.e4m3) return 32;
  const long long most = (long long)a.max_tokens * a.G;
  return may_chunk(a.max_tokens, a.G) && most <= 128 ? 0 : 16;
}

cudaError_t launch_paged_attention(const AttentionArgs& in, cudaStream_t stream) {
  AttentionArgs a = in;
  a.window_rows = window_limit(a);
  // (the workspace holds the chunk kernel's pieces where may_chunk says so)
  const bool chunks = may_chunk(a.max_tokens, a.G) && (long long)a.max_tokens * a.G > a.window_rows;
  // Where T = B max_tokens every request has max_tokens tokens, or some request or offset
  // breaks the contract: the chunk kernel then takes all that are well formed, however short.
  if (chunks && (long long)a.T == (long long)a.B * a.max_tokens) a.window_rows = 0;
  if (a.window_rows > 0) {
    const cudaError_t e = launch_window_attention(a, stream);
    if (e != cudaSuccess || !chunks) return e;
  }
  return launch_chunk_attention(a, stream);
}

}  // namespace kda
