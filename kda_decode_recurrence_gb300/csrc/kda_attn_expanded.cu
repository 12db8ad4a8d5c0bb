// kda_attn_expanded.cu -- latent attention in the expanded form: keys and values per head, for prompts.
//
//   x_j = scale (q_nope . k_j + q_rope . p_j)    128 + 64 entries, p_j shared by the heads
//   o = sum e^(x_j - m) v_j / sum e^(x_j - m),   lse = m + ln sum;   token i of n at position L - n + i
//
// 640 operations per (row, position) on 512 bytes per (position, head) that hundreds of rows share:
// the tensor cores bound it.  A cluster of two CTAs has two slots; each takes a stream of
// items (request, head, 256 tokens), key tiles of 128 positions, with products of the pair
// (cta_group::2, M = 256, each CTA 128 rows):
//   S = Q K^T     256 x 128, contraction 192; a CTA holds 64 of the keys
//   P = 2^(S - m) in bf16 back to tensor memory, by the 128 threads that own a row each
//   O += P V      256 x 128; P from tensor memory, a CTA holds 64 of V's columns, all 128 keys
// (in bf16 because V is, and a product takes one type: 2^-8 of a weight at most, as the output's own rounding;
// errors against 64 bits 0.0020-0.0024, of outputs rounded once 0.0017.  P in two bf16 parts would double PV.)
// While one slot's softmax runs, the other's products do: one warp issues for both, PV of a slot and
// then its next S, in turns.  In a pair a product reads half of B from each SM's shared memory, and
// products with both operands there run at full rate, which a single CTA's do not (S: 64 cycles
// a step of 16 against 107); and each CTA's copies are half.
//
// Streams take even shares of all key tiles; items that are cut are left in pieces for a second kernel.
// O is rescaled only when a row's maximum has grown by more than 2^8.
//
// 2048 new tokens over 6001 before them, 96 heads: 640-673 us by box, 1.31-1.38 PFLOP/s of a cuBLAS product's
// 1.74 held for long (the clock falls to 1.6 GHz under the power limit); 5 prompts of 33-1500, 16 heads: 54 us.
// A slot's chain (S, a row's 128 exponentials, PV) is some 4000 cycles beside 1280 of its products, and two
// of them overlap: tensor cores 57 % of active cycles, exponentials 23 %, issue 33 %.  Of the 4000: 240 until
// S is in registers, 650 to its maximum, 1000 for the weights, 1600 until the next S.
// Measured and left: halves of 64 keys with a product each, P of one beside S of the next (699 us: a step of
// 64 keys takes 43 cycles, of 128 64), two threads to a row (725 us against 664 then), P through shared memory
// with the next S ahead (696 and more), registers dealt by role (651 against 637), kItemCost of 2, 5 and 8.
//
// A key tile that some row sees in part (the diagonal, the end) is masked in the softmax, and entries
// of V that are outside the request, or not finite, are taken out of shared memory first (0 x NaN
// would reach the rows that do not see them); an item that had live entries of that kind adds them,
// for the rows that see them, at its end.
#include <cuda.h>

#include "kda_attn.cuh"
#include "kda_latent.h"
#include "kda_launch.h"
#include "kda_tcgen05.cuh"
#include "kda_tmap.h"

namespace kda {
namespace {

constexpr int kPairs = 76;            // of CTAs, one CTA per SM
constexpr int kStreams = 2 * kPairs;
constexpr int kTile = 128;            // positions per key tile
constexpr int kM = 128;               // rows of an item per CTA
constexpr int kRows = 2 * kM;
constexpr int D = kExpanded, kKeyWidth = kExpanded + kRope;
constexpr int kPanels = kKeyWidth / 64;
constexpr int kQPanel = kM * 128, kKeyPanel = kTile / 2 * 128;  // bytes: 128 rows, 64 keys
constexpr int kKeyBytes = kPanels * kKeyPanel, kValueBytes = kTile * 128;
constexpr int kValues = 2;            // value units kept per slot (of keys: one)
constexpr int kNotes = 4;             // items whose notes are kept
constexpr int kItemCost = 3;          // what an item's beginning and end take, in key tiles
constexpr unsigned long long kPartLimitNs = 60 * kWaitLimitNs;  // limit of a wait for a whole part
constexpr float kGrow = 8.f;          // growth of a maximum (log 2) that rescales O
constexpr float kRounds = 4194304.f;  // maxima past 2^22: half an fp32 step is more than 2^-2
// Warps: 0-3 and 4-7 the slots' softmax, 8 the products, 9 and 10 the slots' copies, 11 passes on values.
constexpr int kMmaWarp = 8, kCopyWarp = 9, kValueWarp = 11, kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kTmemCols = 512, kColO = 256;

// A stream's part of an item; count 0: no more.
struct Part {
  int q0, n, k0, L;   // the request's tokens and keys
  int h, row0;        // head, first row (of the request)
  int tile0, count;
  int whole;          // key tiles that end at or before this position are seen by every row
  int flags;
  int pieces;         // streams that share the item
};
constexpr int kBegins = 1, kEnds = 2;

struct Pairing {  // a request: tokens q0 .. q0 + n - 1, keys k0 .. k0 + L - 1
  int q0, n, k0, L;
};
struct Slot {
  unsigned char q[kPanels][kQPanel];       // this CTA's 128 rows, 1024-aligned, swizzled panels
  unsigned char key[kKeyBytes];            // its 64 keys of a tile
  unsigned char value[kValues][kValueBytes];  // its 64 columns of a tile's values
};

struct Smem {
  Slot slot[2];
  Part part[2][kNotes];
  int bad[2][kNotes];                      // item + 1: live entries of V were taken out of that item
  long long scan[2][kWarps];
  long long first_unit[2];                 // of the requests that hold the streams' first units
  int first_request[2];
  Pairing first[2];                        // they
  uint32_t tmem;
  // this CTA's own (s_full says too that the keys have been read, o_done that the values have)
  uint64_t value_full[2][kValues], s_full[2], o_done[2][kValues], q_empty[2];
  uint64_t part_full[2][kNotes], part_empty[2][kNotes], done;
  // the first CTA's (key_ready, q_ready: both CTAs' copies arrive; the others: both CTAs' warps)
  uint64_t key_ready[2], q_ready[2], value_ready[2][kValues], p_half[2], p_full[2];
};

__device__ __forceinline__ Pairing load_request(const ExpandedArgs& p, int b, bool report) {
  Pairing r;
  r.q0 = fresh(p.cu_q + b);
  r.n = fresh(p.cu_q + b + 1) - r.q0;
  r.k0 = fresh(p.cu_k + b);
  r.L = fresh(p.cu_k + b + 1) - r.k0;
  const bool good = r.q0 >= 0 && r.n >= 0 && r.q0 + (long long)r.n <= p.Tq && r.k0 >= 0 && r.L >= 0 &&
                    r.k0 + (long long)r.L <= p.Tk;
  if (!good) {
    if (report) raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
    r.n = 0;
  }
  return r;
}
__device__ __forceinline__ int row_tiles(const Pairing& r) { return (int)(((long long)r.n + kRows - 1) / kRows); }
// Positions that some row of the tile sees end before this.
__device__ __forceinline__ int tile_end(const ExpandedArgs& p, const Pairing& r, int tile) {
  if (!p.causal) return r.L;
  return min(r.L, max(0, r.L - r.n + (int)min((long long)r.n, (tile + 1ll) * kRows)));
}
// An item's units: what its ends take, and its key tiles (at least one: rows that see nothing are written too).
__device__ __forceinline__ int key_tiles(int end) { return max(1, (end + kTile - 1) / kTile); }
__device__ __forceinline__ int item_units(const ExpandedArgs& p, const Pairing& r, int tile) {
  return kItemCost + key_tiles(tile_end(p, r, tile));
}
// Units of one head of each lane's request: by the lane where there are few row tiles, by the warp
// together where there are many.
__device__ __forceinline__ long long head_units(const ExpandedArgs& p, const Pairing& r, int lane) {
  const int tiles = row_tiles(r);
  const bool many = tiles > 8;
  long long sum = 0;
  if (!many)
    for (int t = 0; t < tiles; ++t) sum += item_units(p, r, t);
  for (unsigned left = __ballot_sync(0xffffffffu, many); left; left &= left - 1) {
    const int src = __ffs(left) - 1;
    Pairing x{0, __shfl_sync(0xffffffffu, r.n, src), 0, __shfl_sync(0xffffffffu, r.L, src)};
    const int all = row_tiles(x);
    long long part = 0;
    for (int t = lane; t < all; t += 32) part += item_units(p, x, t);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == src) sum = part;
  }
  return sum;
}

// The halves of v (two bf16) that are not finite, as a mask.
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  return ((v & 0x7f80u) == 0x7f80u ? 0x0000ffffu : 0u) | ((v & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// Adds the live entries of V that were taken out of an item's partly seen key tiles to columns
// col .. col + 31 of one row's output: the weight of each is found again from Q and K in memory.
// (Rare: values that are not finite.)
__device__ __noinline__ void add_bad_values(const ExpandedArgs& p, size_t q_row, int k0, int h, int from, int to,
                                            float m, int col, float* o) {
  const kda_bf16* q = p.q + q_row * p.q_stride + (size_t)h * kKeyWidth;
  auto value = [](kda_bf16 x) { return __uint_as_float((uint32_t)x << 16); };
  for (int j = from; j < to; ++j) {
    const kda_bf16* k = p.kv + (k0 + j) * p.kv_stride + (size_t)h * (2 * D);
    const kda_bf16* pe = p.k_pe + (k0 + j) * p.pe_stride;
    float w = -1.f;
    for (int d = 0; d < 32; ++d) {
      const kda_bf16 v = k[D + col + d];
      if ((v & 0x7f80u) != 0x7f80u) continue;
      if (w < 0.f) {
        float x = 0.f;
        for (int e = 0; e < D; ++e) x = fmaf(value(q[e]), value(k[e]), x);
        for (int e = 0; e < kRope; ++e) x = fmaf(value(q[D + e]), value(pe[e]), x);
        w = exp2_approx(x * (p.scale * kLog2E) - m);
      }
      o[d] = fmaf(w, value(v), o[d]);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                    const __grid_constant__ CUtensorMap pe_map, const ExpandedArgs p, const Pieces pieces) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.key_ready[t], 1);
      for (int s = 0; s < kValues; ++s) {
        mbar_init(&sm.value_full[t][s], 1);
        mbar_init(&sm.o_done[t][s], 1);
        mbar_init(&sm.value_ready[t][s], 2);
      }
      mbar_init(&sm.q_empty[t], 1);
      mbar_init(&sm.q_ready[t], 1);
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_half[t], 8);
      mbar_init(&sm.p_full[t], 8);
      for (int s = 0; s < kNotes; ++s) {
        mbar_init(&sm.part_full[t][s], 1);
        mbar_init(&sm.part_empty[t][s], rank == 0 ? 6 : 5);  // warps that read notes
        sm.bad[t][s] = 0;
      }
    }
    mbar_init(&sm.done, 1);
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc_pair(&sm.tmem, kTmemCols);
  pdl_wait();
  pdl_trigger();

  // ---- the shares of this pair's streams: a thread counts a request, in passes
  if (blockIdx.x == 0 && tid == 0 &&
      (fresh(p.cu_q) != 0 || fresh(p.cu_q + p.B) != p.Tq || fresh(p.cu_k) != 0 || fresh(p.cu_k + p.B) != p.Tk))
    raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
  if (rank == 0 && tid < 2) pieces.notes[2 * pair + tid].tokens = 0;
  const int passes = (p.B + kThreads - 1) / kThreads;
  long long mine = 0, before = 0, units = 0;
  Pairing r{0, 0, 0, 0};
  for (int i = 0; i < passes; ++i) {
    const int b = i * kThreads + tid;
    r = Pairing{0, 0, 0, 0};
    if (b < p.B) r = load_request(p, b, blockIdx.x == 0);
    mine = p.H * head_units(p, r, lane);
    long long all;
    before = units + scan_before<kWarps>(mine, sm.scan[i & 1], all);
    units += all;
  }
  const int used = (int)min((long long)kStreams, units);
  auto stream_of = [&](int t) { return 2 * pair + t; };
  auto begin_of = [&](int t) { return stream_of(t) < used ? share_begin(units, used, stream_of(t)) : 0; };
  auto end_of = [&](int t) { return stream_of(t) < used ? share_begin(units, used, stream_of(t) + 1) : 0; };
  const long long starts[2] = {begin_of(0), begin_of(1)};
  for (int i = 0; i < passes; ++i) {
    const int b = i * kThreads + tid;
    if (passes > 1) {  // counted again
      if (i == 0) units = 0;
      r = Pairing{0, 0, 0, 0};
      if (b < p.B) r = load_request(p, b, false);
      mine = p.H * head_units(p, r, lane);
      long long all;
      __syncthreads();
      before = units + scan_before<kWarps>(mine, sm.scan[i & 1], all);
      units += all;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (starts[t] >= before && starts[t] < before + mine) {
        sm.first_request[t] = b;
        sm.first_unit[t] = before;
        sm.first[t] = r;
      }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // barriers and tensor memory of both CTAs are there
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  bool ok = true;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && wait_together<true>(smem_u32(bar), parity);
    return ok;
  };
  auto read_part = [&](int t, int item, Part& part) {
    if (!wait(&sm.part_full[t][item % kNotes], (item / kNotes) & 1)) return false;
    part = sm.part[t][item % kNotes];
    return part.count > 0;
  };
  auto leave_part = [&](int t, int item) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.part_empty[t][item % kNotes]);
  };

  if (warp < kMmaWarp) {
    // ---- the softmax: one row per thread
    const int t = warp >> 2, r = tid & (kM - 1);
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = lanes + t * kTile, o_col = lanes + kColO + t * D, p_col = s_col + 64;
    const float c = p.scale * kLog2E;
    const float2 c2 = make_float2(c, c);
    const uint32_t p_half = cluster_addr(&sm.p_half[t], 0), p_full = cluster_addr(&sm.p_full[t], 0);
    int task = 0;
    Part part;
    for (int item = 0; read_part(t, item, part); leave_part(t, item), ++item) {
      const int row = part.row0 + rank * kM + r, pos = part.L - part.n + row;
      const bool live = row < part.n;
      const bool idle = !__any_sync(0xffffffffu, live);  // (what is left in P stays in rows that nobody reads)
      const int row_hi = pos < 0 ? 0 : p.causal ? min(pos + 1, part.L) : part.L;
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      bool rounds = false;  // a maximum of the warp's is past kRounds
      for (int i = 0; i < part.count; ++i, ++task) {
        if (!wait(&sm.s_full[t], task & 1)) break;
        if (idle) {
          if (lane == 0) {
            mbar_arrive_cluster(p_half);
            mbar_arrive_cluster(p_full);
          }
          continue;
        }
        tc_fence_after();
        const int start = (part.tile0 + i) * kTile;
        // whole key tiles take x = c S in one product with the subtraction
        const bool whole = start + kTile <= part.whole;
        const bool plain = whole && c >= 0.f;
        float x[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_32cols(s_col + 32 * q, x[q]);
        tmem_ld_wait();
        // Scores in units of log 2; what is not seen: -infinity.
        auto scored = [&](float(&y)[32], int col) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 a = __fmul2_rn(make_float2(y[e], y[e + 1]), c2);
            y[e] = a.x;
            y[e + 1] = a.y;
          }
          if (!whole) {
            const uint32_t see = columns(0, row_hi - start - col);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1)) y[e] = -INFINITY;
          }
        };
        auto highest = [](const float(&y)[32]) {
          float a = fmaxf(y[0], y[1]), b = fmaxf(y[2], y[3]);
#pragma unroll
          for (int e = 4; e < 32; e += 4) {
            a = max3(a, y[e], y[e + 1]);
            b = max3(b, y[e + 2], y[e + 3]);
          }
          return fmaxf(a, b);
        };
        if (!plain)
#pragma unroll
          for (int q = 0; q < 4; ++q) scored(x[q], 32 * q);
        float top = fmaxf(max3(highest(x[0]), highest(x[1]), highest(x[2])), highest(x[3]));
        if (plain) top *= c;
        // A larger maximum moves the sum and O; S came after the product before it, so O is at rest.
        const float now = fmaxf(m, top);
        if (__any_sync(0xffffffffu, live && now > m + kGrow)) {  // (a row that is not live may hold anything)
          const float keep = exp2_approx(m - (now == -INFINITY ? 0.f : now));
          l2.x *= keep;
          l2.y *= keep;
          if (i > 0) {
#pragma unroll 1
            for (int cc = 0; cc < D; cc += 16) {
              float o[16];
              tmem_ld_16cols(o_col + cc, o);
              tmem_ld_wait();
              uint32_t ob[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) ob[e] = __float_as_uint(o[e] * keep);
              tmem_st_16cols(o_col + cc, ob);
            }
          }
          m = now;
          rounds = __any_sync(0xffffffffu, live && fabsf(m) > kRounds && m != -INFINITY);
        }
        // c S is exact in the one product and the maximum rounded, by hundreds where scores are
        // billions: there both are rounded, so that the largest weight is 1
        const bool fused = plain && !rounds;
        if (__builtin_expect(plain && rounds, 0)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) scored(x[q], 32 * q);
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const float2 nref = make_float2(-ref, -ref);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
        const float2 by = fused ? c2 : make_float2(1.f, 1.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float2 ya = __ffma2_rn(make_float2(x[q][e], x[q][e + 1]), by, nref);
            const float2 yb = __ffma2_rn(make_float2(x[q][e + 2], x[q][e + 3]), by, nref);
            const float2 va = make_float2(exp2_approx(ya.x), exp2_approx(ya.y));
            const float2 vb = make_float2(exp2_approx(yb.x), exp2_approx(yb.y));
            sum0 = __fadd2_rn(sum0, va);
            sum1 = __fadd2_rn(sum1, vb);
            pw[e / 2] = pack_bf16(va.x, va.y);
            pw[e / 2 + 1] = pack_bf16(vb.x, vb.y);
          }
          tmem_st_16cols(p_col + 16 * q, pw);
          if (q & 1) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(q == 1 ? p_half : p_full);
          }
        }
        l2 = __fadd2_rn(l2, __fadd2_rn(sum0, sum1));
      }
      if (!ok || !wait(&sm.o_done[t][(task - 1) % kValues], ((task - 1) / kValues) & 1)) break;
      // ---- the end of this stream's part of the item
      tc_fence_after();
      const float l = l2.x + l2.y;
      const bool done = (part.flags & (kBegins | kEnds)) == (kBegins | kEnds);
      const size_t out_row = (size_t)(part.q0 + row) * p.H + part.h;
      const size_t piece = ((size_t)stream_of(t) * 2 + (part.flags & kBegins ? 1 : 0)) * kRows + rank * kM + r;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool bad = sm.bad[t][item % kNotes] == item + 1;
      if (live) {
        if (!done) pieces.ml[piece] = make_float2(m, l);
        else if (p.lse) p.lse[out_row] = (m + log2f(l)) * kLn2;
      }
      if (rank == 0 && r == 0 && (part.flags & (kBegins | kEnds)) == kBegins)
        pieces.notes[stream_of(t)] =
            PieceNote{part.q0 + part.row0, min(kRows, part.n - part.row0), part.pieces, part.h};
      int to_rows[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) to_rows[e] = __shfl_sync(0xffffffffu, live ? (int)out_row : -1, (lane & ~3) + e);
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 32) {
        float o[32];
        tmem_ld_32cols(o_col + cc, o);
        tmem_ld_wait();
        if (bad && live) {
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = o[e];
          add_bad_values(p, part.q0 + row, part.k0, part.h, max(part.tile0, part.whole / kTile) * kTile,
                         min(row_hi, (part.tile0 + part.count) * kTile), m == -INFINITY ? 0.f : m, cc, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = y[e];
        }
        __syncwarp();
        if (done) {
          uint4 y[4];
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            y[e / 8] = make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                                  pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
          transpose4(y, lane);  // four lanes write 64 bytes of one row together
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (to_rows[e] >= 0)
              *reinterpret_cast<uint4*>(p.out + (size_t)to_rows[e] * D + cc + 8 * (lane & 3)) = y[e];
        } else if (live) {
          // [32 quarters of a row][256 rows]: the lanes of a warp write 512 bytes together
          float4* to = reinterpret_cast<float4*>(pieces.o + (piece - rank * kM - r) * D) + cc / 4 * kRows + rank * kM + r;
#pragma unroll
          for (int e = 0; e < 32; e += 4) to[e / 4 * kRows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        __syncwarp();  // the next load is the whole warp's
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
  } else {
    if (warp == kCopyWarp || warp == kCopyWarp + 1) {
      // ---- a stream's items: their notes, queries, keys and values
      const int t = warp - kCopyWarp;
      Slot& slot = sm.slot[t];
      const long long u0 = starts[t], u1 = end_of(t);
      const uint32_t key_ready = cluster_addr(&sm.key_ready[t], 0), q_ready = cluster_addr(&sm.q_ready[t], 0);
      int key_put = 0, value_put = 0, item = 0;
      auto put_note = [&](const Part& part) {
        // (a part of a very long request may take more than a second)
        if (item >= kNotes)
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&sm.part_empty[t][item % kNotes], (item / kNotes - 1) & 1, kPartLimitNs));
        if (ok && lane == 0) {
          sm.part[t][item % kNotes] = part;
          mbar_arrive(&sm.part_full[t][item % kNotes]);
        }
        __syncwarp();
      };
      long long unit = 0;
      int b = 0, h = 0, tile = 0, tiles = 0, base = 0;
      Pairing r{0, 0, 0, 0}, held{0, 0, 0, 0};  // held: request base + lane
      auto fetch = [&]() {
        base = b;
        held = Pairing{0, 0, 0, 0};
        if (b + lane < p.B) held = load_request(p, b + lane, false);
      };
      auto take = [&]() {  // the first request from b on that has rows
        while (b < p.B) {
          if (b >= base + 32) fetch();
          const unsigned some = __ballot_sync(0xffffffffu, held.n > 0) & (0xffffffffu << (b - base));
          if (some) {
            const int src = __ffs(some) - 1;
            b = base + src;
            r.q0 = __shfl_sync(0xffffffffu, held.q0, src);
            r.n = __shfl_sync(0xffffffffu, held.n, src);
            r.k0 = __shfl_sync(0xffffffffu, held.k0, src);
            r.L = __shfl_sync(0xffffffffu, held.L, src);
            h = tile = 0;
            tiles = row_tiles(r);
            return;
          }
          b = base + 32;
        }
      };
      if (u1 > u0) {
        b = sm.first_request[t];
        unit = sm.first_unit[t];
        r = sm.first[t];
        tiles = row_tiles(r);
        base = b - 32;  // (the requests after it are fetched when they are wanted)
        // the head and the row tile that hold u0
        const long long each = __shfl_sync(0xffffffffu, head_units(p, r, lane), 0);
        h = (int)((u0 - unit) / each);
        unit += h * each;
        while (true) {
          const int x = tile + lane < tiles ? item_units(p, r, tile + lane) : 0;
          long long upto = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          const unsigned past = __ballot_sync(0xffffffffu, unit + upto > u0);
          if (past || tile + 32 >= tiles) {
            const int in = past ? __ffs(past) - 1 : 0;
            unit += __shfl_sync(0xffffffffu, upto - x, in);
            tile += in;
            break;
          }
          unit += __shfl_sync(0xffffffffu, upto, 31);
          tile += 32;
        }
      }
      while (u1 > u0 && unit < u1 && b < p.B && ok) {
        const int all = key_tiles(tile_end(p, r, tile));
        const int from = (int)max(0ll, u0 - unit - kItemCost), to = (int)min((long long)all, u1 - unit - kItemCost);
        if (to > from) {
          Part part;
          part.q0 = r.q0;
          part.n = r.n;
          part.k0 = r.k0;
          part.L = r.L;
          part.h = h;
          part.row0 = tile * kRows;
          part.tile0 = from;
          part.count = to - from;
          const int first = r.L - r.n + part.row0;
          part.whole = p.causal ? max(0, first + 1) : first >= 0 ? r.L : 0;
          part.flags = (from == 0 ? kBegins : 0) | (to == all ? kEnds : 0);
          part.pieces = to == all ? 1 : share_of(units, used, unit + kItemCost + all - 1) - stream_of(t) + 1;
          put_note(part);
          if (item > 0) wait(&sm.q_empty[t], (item - 1) & 1);
          ++item;
          if (!ok) break;
          if (rank == 0 && lane == 0) mbar_expect_tx(&sm.q_ready[t], 2 * kPanels * kQPanel);
          __syncwarp();
          if (lane < kPanels)
            tma_load_3d_pair(slot.q[lane], &q_map, q_ready, lane * 64, h, r.q0 + part.row0 + rank * kM);
          for (int i = 0; i < part.count; ++i) {
            // this CTA's half of the keys; both CTAs' copies arrive at the first's barrier
            const int v = value_put % kValues, at = r.k0 + (from + i) * kTile;
            if (key_put > 0) wait(&sm.s_full[t], (key_put - 1) & 1);
            if (!ok) break;
            ++key_put;
            if (rank == 0 && lane == 0) mbar_expect_tx(&sm.key_ready[t], 2 * kKeyBytes);
            __syncwarp();
            const int mine = at + rank * (kTile / 2);
            if (lane < 2) tma_load_3d_pair(slot.key + lane * kKeyPanel, &kv_map, key_ready, lane * 64, h, mine);
            else if (lane == 2) tma_load_3d_pair(slot.key + 2 * kKeyPanel, &pe_map, key_ready, 0, 0, mine);
            // its columns of all values
            if (value_put >= kValues) wait(&sm.o_done[t][v], (value_put / kValues - 1) & 1);
            if (!ok) break;
            ++value_put;
            if (lane == 0) mbar_expect_tx(&sm.value_full[t][v], kValueBytes);
            __syncwarp();
            if (lane < 2)
              tma_load_3d(slot.value[v] + lane * kKeyPanel, &kv_map, &sm.value_full[t][v], D + rank * 64, h,
                          at + lane * (kTile / 2));
          }
        }
        unit += kItemCost + all;
        if (++tile >= tiles) {
          tile = 0;
          if (++h >= p.H) {
            ++b;
            take();
          }
        }
      }
      if (ok) put_note(Part{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0});
      if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
      // Every copy lands before the CTA's memory is released, also when a wait gave up (keys and queries: the
      // first CTA waits for both).
      for (int u = max(0, value_put - kValues); u < value_put; ++u)
        mbar_wait(&sm.value_full[t][u % kValues], (u / kValues) & 1);
      if (rank == 0) {
        if (key_put > 0) mbar_wait(&sm.key_ready[t], (key_put - 1) & 1);
        if (item > 0) mbar_wait(&sm.q_ready[t], (item - 1) & 1);
      }
    } else if (warp == kMmaWarp && rank == 0) {
      // ---- the products of both slots
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t idesc_s = idesc_bf16(kTile, kRows, false, false), idesc_o = idesc_bf16(D, kRows, false, true);
      // A slot's items begun, key tiles of the last one left, key tiles whose PV has been issued; whether an S
      // is under way (then its PV comes next), the item's first one.
      struct State {
        int item, left, tasks;
        bool live, first;
      };
      State here{0, 0, 0, true, false}, there{0, 0, 0, true, false};  // slot t's, the other's
      const uint32_t one = elect_one() ? 1u : 0u;
      auto scores = [&](int t) {  // the slot's next S
        here.live = false;
        if (here.left == 0) {
          if (here.item > 0) leave_part(t, here.item - 1);
          Part part;
          if (!read_part(t, here.item, part)) return;
          here.left = __shfl_sync(0xffffffffu, part.count, 0);
          here.first = true;
          wait(&sm.q_ready[t], here.item & 1);
          ++here.item;
        }
        if (!wait(&sm.key_ready[t], here.tasks & 1)) return;
        tc_fence_after();
        --here.left;
        const uint64_t a = smem_desc_sw128(smem_u32(sm.slot[t].q[0]), 16, 1024);
        const uint64_t k = smem_desc_sw128(smem_u32(sm.slot[t].key), 16, 1024);
#pragma unroll
        for (int j = 0; j < kKeyWidth / 16; ++j)  // 32 bytes on, or the next panel
          mma_bf16_pair_if(one, base + t * kTile, a + (j & 3) * 2 + (j >> 2) * (kQPanel / 16),
                           k + (j & 3) * 2 + (j >> 2) * (kKeyPanel / 16), idesc_s, j > 0 ? 1u : 0u);
        mma_commit_pair_if(one, &sm.s_full[t]);
        if (here.left == 0) mma_commit_pair_if(one, &sm.q_empty[t]);
        here.live = true;
      };
      auto output = [&](int t) {  // PV of the slot's S under way
        const int s = here.tasks % kValues;
        const uint32_t d = base + kColO + t * D, pc = base + t * kTile + 64;
        const uint64_t v = smem_desc_sw128(smem_u32(sm.slot[t].value[s]), kTile * 128, 1024);
        wait(&sm.value_ready[t][s], (here.tasks / kValues) & 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait(half ? &sm.p_full[t] : &sm.p_half[t], here.tasks & 1)) return;
          tc_fence_after();
#pragma unroll
          for (int j = 4 * half; j < 4 * half + 4; ++j)
            mma_bf16_pair_tmem_a_if(one, d, pc + 8 * j, v + ((j * 16 * 128) >> 4), idesc_o,
                                    !here.first || j > 0 ? 1u : 0u);
        }
        mma_commit_pair_if(one, &sm.o_done[t][s]);
        here.first = false;
        ++here.tasks;
      };
#pragma unroll 1
      for (int step = 0; ok && (here.live || there.live); ++step) {
        const int t = __shfl_sync(0xffffffffu, step & 1, 0);
        if (here.live) {
          if (step > 1) output(t);
          if (ok) scores(t);
        }
        const State x = here;
        here = there;
        there = x;
      }
      if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
      mma_commit_pair_if(one, &sm.done);  // arrives when every product issued has completed
      mbar_wait(&sm.done, 0);
    } else if (warp == kValueWarp) {
      // ---- values that have arrived, without the entries that some row must not see; both slots' in
      // the order of their arrival
      const uint32_t ready[2] = {cluster_addr(sm.value_ready[0], 0), cluster_addr(sm.value_ready[1], 0)};
      Part part[2];
      int item[2] = {0, 0}, at[2] = {0, 0}, tasks[2] = {0, 0};
      bool have[2] = {false, false}, over[2] = {false, false};
      unsigned long long since = global_ns();
      auto there = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(smem_u32(bar), parity)); };
      while (ok && !(over[0] && over[1])) {
        bool moved = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!over[t] && !have[t] && there(&sm.part_full[t][item[t] % kNotes], (item[t] / kNotes) & 1)) {
            part[t] = sm.part[t][item[t] % kNotes];
            over[t] = part[t].count == 0;
            have[t] = !over[t];
            at[t] = 0;
            moved = true;
          }
          const int s = tasks[t] % kValues;
          if (have[t] && there(&sm.value_full[t][s], (tasks[t] / kValues) & 1)) {
            const int start = (part[t].tile0 + at[t]) * kTile;
            if (start + kTile > part[t].whole) {
              unsigned char* v = sm.slot[t].value[s];
              const int to = part[t].L - start;  // the request's keys
              auto chunk = [&](int i) { return reinterpret_cast<uint4*>(v + swizzled<128>(i >> 3, i & 7)); };
              if (to < kTile) {
#pragma unroll 1
                for (int i = max(0, to) * 8 + lane; i < kTile * 8; i += 32) *chunk(i) = make_uint4(0, 0, 0, 0);
                __syncwarp();
              }
              // 0 x is 0 for all that is finite, so that a sum tells
              const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
              __nv_bfloat162 sum[4] = {zero, zero, zero, zero};
#pragma unroll 1
              for (int first = lane; first < kTile * 8; first += 8 * 32) {
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = *chunk(first + 32 * i);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  sum[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[i].x), zero, sum[0]);
                  sum[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[i].y), zero, sum[1]);
                  sum[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[i].z), zero, sum[2]);
                  sum[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[i].w), zero, sum[3]);
                }
              }
              const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
              if (__any_sync(0xffffffffu, __hisnan(all.x) || __hisnan(all.y))) {
#pragma unroll 1
                for (int i = lane; i < kTile * 8; i += 32) {
                  const uint4 x = *chunk(i);
                  const uint4 out = make_uint4(not_finite(x.x), not_finite(x.y), not_finite(x.z), not_finite(x.w));
                  if (out.x | out.y | out.z | out.w)
                    *chunk(i) = make_uint4(x.x & ~out.x, x.y & ~out.y, x.z & ~out.z, x.w & ~out.w);
                }
                // the rows of either CTA add them at the item's end
                if (lane == 0)
                  for (int to = 0; to < 2; ++to)
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&sm.bad[t][item[t] % kNotes], to)),
                                 "r"(item[t] + 1)
                                 : "memory");
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(ready[t] + 8 * s);
            ++tasks[t];
            if (++at[t] == part[t].count) {
              leave_part(t, item[t]++);
              have[t] = false;
            }
            moved = true;
          }
        }
        if (moved) since = global_ns();
        else if (__any_sync(0xffffffffu, global_ns() - since > kWaitLimitNs)) ok = false;
      }
      if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // nothing of the pair is under way
  tc_fence_after();
  if (warp == kMmaWarp) {
    mbar_wait<true>(&sm.done, 0);  // (the second CTA's word of it)
    __syncwarp();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
  __syncwarp();
  cluster_sync();
}

// The pieces of one shared item into its outputs: with m = max m_i,
//   o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i,   lse = (m + log2 l) ln 2.
// CTA (c, y) takes 16 columns from 16 (y / 2) on of 128 rows, y % 2, in the item that stream c began.
constexpr int kJoinY = 2 * D / 16;
__global__ void __launch_bounds__(128) expanded_join_kernel(const ExpandedArgs p, const Pieces s) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, cc = blockIdx.y >> 1, row = (blockIdx.y & 1) * 128 + threadIdx.x;
  const PieceNote note = s.notes[c];
  if (row >= note.tokens) return;
  auto at = [&](int i) { return ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * kRows; };
  float m = -INFINITY, l = 0.f;
  float4 o[4] = {};
#pragma unroll 2
  for (int i = 0; i < note.pieces; ++i) {
    const float2 ml = s.ml[at(i) + row];
    const float4* from = reinterpret_cast<const float4*>(s.o + at(i) * D) + cc * 4 * kRows + row;
    float4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = from[e * kRows];
    const float now = fmaxf(m, ml.x), ref = now == -INFINITY ? 0.f : now;
    const float keep = exp2_approx(m - ref), w = exp2_approx(ml.x - ref);
    m = now;
    l = fmaf(w, ml.y, l * keep);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e].x = fmaf(w, x[e].x, o[e].x * keep);
      o[e].y = fmaf(w, x[e].y, o[e].y * keep);
      o[e].z = fmaf(w, x[e].z, o[e].z * keep);
      o[e].w = fmaf(w, x[e].w, o[e].w * keep);
    }
  }
  const size_t out_row = (size_t)(note.row0 + row) * p.H + note.head;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint4* to = reinterpret_cast<uint4*>(p.out + out_row * D + 16 * cc);
#pragma unroll
  for (int e = 0; e < 4; e += 2)
    to[e / 2] = make_uint4(pack_bf16(o[e].x * inv, o[e].y * inv), pack_bf16(o[e].z * inv, o[e].w * inv),
                           pack_bf16(o[e + 1].x * inv, o[e + 1].y * inv), pack_bf16(o[e + 1].z * inv, o[e + 1].w * inv));
  if (p.lse && cc == 0) p.lse[out_row] = (m + log2f(l)) * kLn2;
}

}  // namespace

size_t expanded_workspace_bytes(int B, int Tq, int H) {
  if (B < 0 || Tq < 0 || H < 1) return 0;
  return (pieces_bytes(kStreams, kRows, D) + 255) & ~(size_t)255;
}

cudaError_t launch_latent_expanded(const ExpandedArgs& a, cudaStream_t stream) {
  static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "a CTA fits an SM");
  CUtensorMap q_map, kv_map, pe_map;
  auto q_like = [&](CUtensorMap* map, int rows) {
    return make_map_3d_bf16(map, a.q, kKeyWidth, a.H, a.Tq, kKeyWidth * 2, (uint64_t)a.q_stride * 2, 64, 1, rows);
  };
  if (!q_like(&q_map, kM)) return cudaErrorInvalidValue;
  if (a.Tk == 0) {  // no rows to make maps of: any will do, nobody sees a key
    if (!q_like(&kv_map, kTile / 2) || !q_like(&pe_map, kTile / 2)) return cudaErrorInvalidValue;
  } else if (!make_map_3d_bf16(&kv_map, a.kv, 2 * D, a.H, a.Tk, 2 * D * 2, (uint64_t)a.kv_stride * 2, 64, 1, kTile / 2) ||
             !make_map_3d_bf16(&pe_map, a.k_pe, kRope, 1, a.Tk, kRope * 2, (uint64_t)a.pe_stride * 2, 64, 1, kTile / 2)) {
    return cudaErrorInvalidValue;
  }
  const size_t smem = sizeof(Smem) + 1024;
  static SmemSet set;
  cudaError_t e = allow_smem(expanded_kernel, smem, set);
  if (e != cudaSuccess) return e;
  const Pieces pieces = pieces_at(a.workspace, kStreams, kRows);
  e = launch_pairs(expanded_kernel, dim3(2 * kPairs), dim3(kThreads), smem, stream, q_map, kv_map, pe_map, a, pieces);
  if (e != cudaSuccess) return e;
  return launch(expanded_join_kernel, dim3(kStreams, kJoinY), dim3(128), 0, stream, true, a, pieces);
}

}  // namespace kda
