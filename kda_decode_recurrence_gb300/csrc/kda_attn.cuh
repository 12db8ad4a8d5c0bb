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

constexpr int kWindowCtas = 456;  // three per SM of a GB300 at most
constexpr int kChunkCtas = 152;   // one per SM
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
  r.t0 = fresh(p.cu + b);
  r.n = fresh(p.cu + b + 1) - r.t0;
  r.L = fresh(p.lens + b);
  const bool good = r.t0 >= 0 && r.n >= 0 && r.t0 + (long long)r.n <= p.T && r.n <= p.max_tokens &&
                    r.L >= 0 && r.L <= (long long)p.c.max_pages * p.c.page_size;
  if (!good) {
    if (report) raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
    r.n = 0;
  }
  return r;
}

// By one thread of the call: offsets that do not span the T tokens are reported (rows outside
// them are nobody's and stay as they are).
__device__ __forceinline__ void check_offsets(const AttentionArgs& p) {
  if (fresh(p.cu) != 0 || fresh(p.cu + p.B) != p.T) raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
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

inline size_t pieces_bytes(int ctas, int rows, int D) {
  return ctas * (sizeof(PieceNote) + 2 * (size_t)rows * (sizeof(float2) + D * sizeof(float)));
}
inline Pieces pieces_at(void* base, int ctas, int rows) {
  Pieces s;
  s.notes = static_cast<PieceNote*>(base);
  s.ml = reinterpret_cast<float2*>(s.notes + ctas);
  s.o = reinterpret_cast<float*>(s.ml + (size_t)ctas * 2 * rows);
  return s;
}

// Byte offset of 16-byte chunk c of row r in a panel of kPanelBytes rows under TMA's
// 128- or 64-byte swizzle.
template <int kPanelBytes>
__device__ __forceinline__ int swizzled(int r, int c) {
  return kPanelBytes == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Two e4m3 codes, one in the high byte of each half of x (low bytes 0), as bf16 values:
// s eeee mmm becomes a bf16 of exponent field eeee, 2^-120 too small (subnormal
// codes and bf16 subnormals alike), and one exact product puts that right.
__device__ __forceinline__ uint32_t widen(uint32_t x) {
  const uint32_t y = (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x7b807b80u));  // 2^120, twice
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Sum of x over the CTA's threads before this one, and over all; kWarps warps, `part`
// in shared memory (one entry a warp).
template <int kWarps>
__device__ __forceinline__ long long scan_before(long long x, long long* part, long long& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long scan = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += y;
  }
  if (lane == 31) part[warp] = scan;
  __syncthreads();
  long long before = scan - x;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += part[w];
    all += part[w];
  }
  return before;
}

// Rows (tokens x G) up to which a request of the call is the window kernel's.
int window_limit(const AttentionArgs& a);
// Rows of its variant that holds every such request of at most max_tokens tokens.
int window_rows(int max_tokens, int G);
cudaError_t launch_window_attention(const AttentionArgs& a, cudaStream_t stream);

constexpr int kChunkRows = 256;  // rows of an item of the chunk kernel, which takes the other requests
cudaError_t launch_chunk_attention(const AttentionArgs& a, cudaStream_t stream);

cudaError_t launch_join_pieces(const AttentionArgs& a, const Pieces& pieces, int rows, int ctas,
                               cudaStream_t stream);

}  // namespace kda
