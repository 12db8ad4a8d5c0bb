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
  int row0;     // first row of the item's outputs: token * H + first head (expanded: its first token)
  int tokens;   // its tokens (absorbed: its rows; 0: this CTA begins no shared item)
  int pieces;   // CTAs, pairs or streams that share it
  int head;     // expanded: its head
};

struct Pieces {
  PieceNote* notes;
  float2* ml;   // [ctas][2][rows]: maximum (in units of log 2), sum
  float* o;     // [ctas][2][rows x D], a piece's in the order in which its kernel's threads hold them
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The bits of columns lo .. hi - 1 among columns 0 .. 31.
__device__ __forceinline__ uint32_t below(int k) { return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u; }
__device__ __forceinline__ uint32_t columns(int lo, int hi) { return below(hi) & ~below(lo); }

// Drafted trees: which of 32 positions a new token sees, the first being a positions behind the
// cached ones (a < 0: before their end).  words: the token's mask, bit i of word w for new token
// 32 w + i of its request, which has n (at most 32 mask_words).
__device__ __forceinline__ uint32_t tree_bits(const int32_t* words, int mask_words, int n, int a) {
  const int w = a >> 5;
  const uint32_t lo = w < 0 ? 0xffffffffu : w < mask_words ? (uint32_t)words[w] : 0u;
  const uint32_t hi = w + 1 < 0 ? 0xffffffffu : w + 1 < mask_words ? (uint32_t)words[w + 1] : 0u;
  return __funnelshift_r(lo, hi, a & 31) & below(n - a);
}

// Lanes 4 i .. 4 i + 3: x[e] of lane j becomes x[j] of lane e.
__device__ __forceinline__ void transpose4(uint4 (&x)[4], int lane) {
#pragma unroll
  for (int bit = 1; bit < 4; bit *= 2) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
      uint4& lo = x[i];
      uint4& hi = x[i + bit];
      uint4 y = up ? lo : hi;
      y.x = __shfl_xor_sync(0xffffffffu, y.x, bit);
      y.y = __shfl_xor_sync(0xffffffffu, y.y, bit);
      y.z = __shfl_xor_sync(0xffffffffu, y.z, bit);
      y.w = __shfl_xor_sync(0xffffffffu, y.w, bit);
      if (up) lo = y;
      else hi = y;
    }
  }
}

// A wait of a whole warp; what follows when the phase is not there at once is out of
// line, so that the product warps' waits take little room in the instruction cache.
template <bool kCluster = false>
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = global_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (__all_sync(0xffffffffu, mbar_try<kCluster>(bar, parity))) return true;
    if (__any_sync(0xffffffffu, global_ns() - t0 > kWaitLimitNs)) return false;
  }
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait_together(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_try<kCluster>(bar, parity)) || wait_on<kCluster>(bar, parity);
}

// A role's share of the registers that the block was launched with.
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
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
