// kda_attn.cuh -- what the attention kernels share: a request's new tokens and the
// positions they see, the even division of all (row tile, key tile) pairs over the
// CTAs, and the pieces in which an item that was divided is left to be joined.
//
// An item is one row tile of one (request, key head); its units are the key tiles its
// rows see.  All units of a call, in the order (request, row tile, key head, key
// tile), are divided evenly over the CTAs: CTA c takes units c U / C .. (c + 1) U / C.
// A CTA finishes the items that lie wholly in its range and leaves a piece
// (unnormalised output, maximum, sum per row) of an item that it shares: at
// most one that began before its range (place 0) and one that it begins
// (place 1).  The join kernel starts at each place 1.
#pragma once

#include "kda_async.cuh"
#include "kda_common.cuh"
#include "kda_paged.h"

namespace kda {

constexpr int kMaxAttnCtas = 304;  // two per SM of a GB300
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A request's new tokens t0 .. t0 + n - 1 and its length; n = 0: nothing to do.
struct Request {
  int t0, n, L;
};

// `report`: raise the status bit of a malformed request (one CTA does).
__device__ __forceinline__ Request load_request(const AttentionArgs& p, int b, bool report) {
  Request r;
  r.t0 = __ldg(p.cu + b);
  r.n = __ldg(p.cu + b + 1) - r.t0;
  r.L = __ldg(p.lens + b);
  const bool good = r.t0 >= 0 && r.n >= 0 && r.t0 + (long long)r.n <= p.T && r.n <= p.max_tokens &&
                    r.L >= 0 && r.L <= (long long)p.c.max_pages * p.c.page_size;
  if (!good) {
    if (report) raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
    r.n = 0;
  }
  return r;
}

// Positions [lo, hi) that the token at position pos sees (none for padding, pos < 0).
__device__ __forceinline__ int seen_lo(const AttentionArgs& p, int pos) {
  return p.window > 0 ? max(0, pos - p.window + 1) : 0;
}
__device__ __forceinline__ int seen_hi(const AttentionArgs& p, int pos, int L) {
  return pos < 0 ? 0 : p.causal ? pos + 1 : L;
}

// CTA c's share of `units`: from unit share_begin(c) to share_begin(c + 1) - 1, and
// the CTA whose share holds unit u.
__device__ __forceinline__ long long share_begin(long long units, int ctas, int c) {
  return units * c / ctas;
}
__device__ __forceinline__ int share_of(long long units, int ctas, long long u) {
  return (int)(((u + 1) * ctas - 1) / units);
}

// Pieces in the workspace: per CTA a note of the item it begins but does not
// finish, then per CTA and place kRows maxima and sums, then kRows x D outputs.
struct PieceNote {
  int row0;     // first row of the item's outputs: token * H + first head
  int tokens;   // its tokens (0: this CTA begins no shared item)
  int pieces;   // CTAs that share it
  int pad;
};

struct Pieces {
  PieceNote* notes;
  float2* ml;   // [ctas][2][rows]: maximum (in units of log 2), sum
  float* o;     // [ctas][2][rows][D]
};

__host__ __device__ inline size_t pieces_bytes(int rows, int D) {
  return kMaxAttnCtas * (sizeof(PieceNote) + 2 * (size_t)rows * (sizeof(float2) + D * sizeof(float)));
}
__host__ __device__ inline Pieces pieces_at(void* base, int rows) {
  Pieces s;
  s.notes = static_cast<PieceNote*>(base);
  s.ml = reinterpret_cast<float2*>(s.notes + kMaxAttnCtas);
  s.o = reinterpret_cast<float*>(s.ml + (size_t)kMaxAttnCtas * 2 * rows);
  return s;
}

constexpr int kWindowRows = 64;  // rows (tokens x G) of a request that the window kernel takes
int window_rows(int max_tokens, int G);
cudaError_t launch_window_attention(const AttentionArgs& a, cudaStream_t stream);

cudaError_t launch_join_pieces(const AttentionArgs& a, const Pieces& pieces, int rows, int ctas,
                               cudaStream_t stream);

}  // namespace kda
