// kda_attn_tree_pairs.cu -- attention of drafted trees over a paged K/V cache, heads of 128.
//
//   A request's new tokens are the nodes of a tree; a node sees every position before the tree and
//   the nodes that its mask names.  x_j = scale q . k_j,  o = sum e^(x_j - m) v_j / sum e^(x_j - m),
//   lse = m + ln sum, rows i G + g for node i and head g of a key head's group.
//
// Some hundred rows (nodes x query heads per key head) share a key head's rows: over bf16 HBM and the
// tensor cores bound a call about equally.  A cluster of two CTAs has two slots, each with a
// stream of items (request, up to 2 (128 / G) nodes, key head), key tiles of 128 positions, with
// products of the pair (cta_group::2, M = 256, each CTA 128 rows, half of the keys for S and half of V's
// columns for PV): S and P share tensor memory, one warp issues for both slots in turns.
// P is in bf16 because V is, and a product takes one type: 2^-8 of a weight at most, as the output's own rounding
// (errors against 64 bits 0.0019-0.0024, of outputs rounded once 0.0017).
// Over e4m3 two warps a slot widen the codes to bf16 on the way (exactly), each CTA its half: a key's scale
// multiplies its column of S, a value's its column of P before the rounding.
//
// Streams take even shares of all key tiles; items that are cut are left in pieces for a second kernel.
//
// 32 trees of 8-60 nodes over 1000-8000, 32 / 8 heads, bf16: 130-133 us by box, 4.3-4.4 TB/s of cache (the chunk
// kernel with masks: 134); 16 of 4-32 over 500-12000, 96 / 8 heads, e4m3: 196 us (270); one of 13 nodes over 517: 16 us.
// A slot's chain (S, a row's 128 exponentials, PV) is some 4000 cycles of a key tile beside 1024 of its
// products, and two of them overlap: 16 trees of 60 nodes over 4060: DRAM 54 %, tensor cores 49 %.  e4m3 adds two
// products per pair of scores; without the codes' widening the 194 us would be 187, with one scale less 181-183.
// Measured and left: an item's nodes dealt evenly to the two CTAs (128 -> 130 us), e4m3's S read twice from tensor
// memory in place of 128 registers (194 -> 216), kItemCost of 1, 2 and 5.
//
// In key tiles with nodes, or the sequence's end, scores are masked, and entries of V that are not the
// request's, or not finite, are taken out of shared memory first (0 x NaN would reach the rows that do not
// see them); an item that had live entries of that kind adds them, for the rows that see them, at its end.
// (e4m3 codes are finite; their scales may not be, and the weights of what a row does not see stay 0.)
#include <cuda.h>

#include "kda_attn.cuh"
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
constexpr int D = 128;
constexpr int kPanels = D / 64;
constexpr int kQPanel = kM * 128, kKeyPanel = kTile / 2 * 128;  // bytes: 128 rows, 64 keys
constexpr int kKeyBytes = kPanels * kKeyPanel, kValueBytes = kTile * 128;
constexpr int kRawBytes = kTile / 2 * D;  // a CTA's codes of a tile, of keys or of values
constexpr int kRing = 2;              // key tiles whose keys and values are kept per slot (e4m3: codes)
constexpr int kScales = 4;            // key tiles whose scales are kept
constexpr int kNotes = 4;             // items whose notes are kept
constexpr int kItemCost = 3;          // what an item's beginning and end take, in key tiles
constexpr unsigned long long kPartLimitNs = 60 * kWaitLimitNs;  // limit of a wait for a whole part
// Warps: 0-3 and 4-7 the slots' softmax, 8 the products, 9 and 10 the slots' copies, 12-13 and 14-15 what is
// done to the slots' copies before the products (11 makes up a warpgroup).
constexpr int kMmaWarp = 8, kCopyWarp = 9, kPrepareWarp = 12, kWarps = 16;
constexpr int kThreads = 32 * kWarps;
// Registers per thread: 65536 at launch, then dealt by role.  (16 trees of 4-32 nodes over 500-12000
// positions of e4m3, 96 heads to 8: 184 for the softmax 211 us, 192 200, 200 194; bf16 takes them all alike.)
constexpr int kSoftmaxRegs = 200, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= 65536, "they fit in the launch's");
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr float kGrow = 8.f;          // growth of a maximum (log 2) that rescales O
constexpr float kRounds = 4194304.f;  // maxima past 2^22: half an fp32 step is more than 2^-2

// A stream's part of an item; count 0: no more.
struct Part {
  int b, t0, n, L;
  int h, token0;      // key head, first node (of the request)
  int tile0, count;
  int flags;
  int pieces;         // streams that share the item
};
constexpr int kBegins = 1, kEnds = 2;

template <bool kE4m3>
struct alignas(1024) Slot {
  unsigned char q[kPanels][kQPanel];       // this CTA's 128 rows, 1024-aligned, swizzled panels
  unsigned char key[kE4m3 ? 1 : kRing][kKeyBytes];      // its 64 keys of a tile
  unsigned char value[kE4m3 ? 1 : kRing][kValueBytes];  // its 64 columns of a tile's values
  unsigned char raw_key[kE4m3 ? kRing : 1][kE4m3 ? kRawBytes : 16];
  unsigned char raw_value[kE4m3 ? kRing : 1][kE4m3 ? kRawBytes : 16];
  float scale[kE4m3 ? kScales : 1][2][kE4m3 ? kTile : 4];  // of all keys (times the softmax's) and values of a tile
};

template <bool kE4m3>
struct TreeSmem {
  Slot<kE4m3> slot[2];
  Part part[2][kNotes];
  int bad[2][kNotes];                      // item + 1: live entries of V were taken out of that item
  long long scan[2][kWarps];
  long long first_unit[2];                 // of the requests that hold the streams' first units
  int first_request[2];
  uint32_t tmem;
  // this CTA's own (s_full says too that the keys have been read, o_done that the values have)
  uint64_t key_full[2][kRing], value_full[2][kRing], key_free[2][kRing], value_free[2][kRing];
  uint64_t s_full[2][kRing], o_done[2][kRing], q_empty[2], part_full[2][kNotes], part_empty[2][kNotes], done;
  // the first CTA's
  uint64_t key_ready[2][kRing], value_ready[2][kRing], q_ready[2], p_half[2], p_full[2];
};

// An item's units: what its ends take, and its key tiles (at least one: rows that see nothing are written too).
__device__ __forceinline__ int key_tiles(int L) { return max(1, (L + kTile - 1) / kTile); }
__device__ __forceinline__ long long tree_units(const AttentionArgs& p, const Request& r, int nodes) {
  return (long long)((r.n + nodes - 1) / nodes) * p.c.HKV * (kItemCost + key_tiles(r.L));
}

// The halves of v (two bf16) that are not finite, as a mask.
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  return ((v & 0x7f80u) == 0x7f80u ? 0x0000ffffu : 0u) | ((v & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// Adds the live entries of V that were taken out of an item's key tiles from position `from` on to columns
// col .. col + 31 of one row's output: the weight of each is found again from Q and K in memory.
// (Rare: values that are not finite, of a bf16 cache; e4m3 codes are finite.)
__device__ __noinline__ void add_bad_nodes(const AttentionArgs& p, int b, int h, int L, int n, int from, int to,
                                           const int32_t* words, const kda_bf16* q, float m, int col, float* o) {
  const kda_bf16* k = static_cast<const kda_bf16*>(p.c.k);
  const kda_bf16* v = static_cast<const kda_bf16*>(p.c.v);
  const int32_t* table = p.c.page_table + (size_t)b * p.c.max_pages;
  for (int j = from; j < to; ++j) {
    if (!(tree_bits(words, p.tree_words, n, j - (L - n)) & 1)) continue;
    const int page = table[j / p.c.page_size];
    if (page < 0 || page >= p.c.num_pages) continue;
    const size_t row = ((size_t)page * p.c.HKV + h) * p.c.page_size + j % p.c.page_size;
    float w = -1.f;
    for (int d = 0; d < 32; ++d) {
      const float value = __uint_as_float((uint32_t)v[row * D + col + d] << 16);
      if (isfinite(value)) continue;
      if (w < 0.f) {
        float x = 0.f;
        for (int e = 0; e < D; ++e)
          x = fmaf(__uint_as_float((uint32_t)q[e] << 16), __uint_as_float((uint32_t)k[row * D + e] << 16), x);
        w = exp2_approx(x * (p.scale * kLog2E) - m);
      }
      o[d] = fmaf(w, value, o[d]);
    }
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map, const AttentionArgs p, const Pieces pieces) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  TreeSmem<kE4m3>& sm =
      *reinterpret_cast<TreeSmem<kE4m3>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1;
  const int per_cta = kM / p.G, nodes = 2 * per_cta;  // nodes of an item

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&sm.key_full[t][s], 1);
        mbar_init(&sm.value_full[t][s], 1);
        mbar_init(&sm.key_free[t][s], 2);
        mbar_init(&sm.value_free[t][s], 2);
        mbar_init(&sm.s_full[t][s], 1);
        mbar_init(&sm.o_done[t][s], 1);
        mbar_init(&sm.key_ready[t][s], kE4m3 ? 4 : 1);
        mbar_init(&sm.value_ready[t][s], 4);
      }
      mbar_init(&sm.q_empty[t], 1);
      mbar_init(&sm.q_ready[t], 1);
      mbar_init(&sm.p_half[t], 8);
      mbar_init(&sm.p_full[t], 8);
      for (int s = 0; s < kNotes; ++s) {
        mbar_init(&sm.part_full[t][s], 1);
        mbar_init(&sm.part_empty[t][s], rank == 0 ? 7 : 6);  // warps that read notes
        sm.bad[t][s] = 0;
      }
    }
    mbar_init(&sm.done, 1);
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc_pair(&sm.tmem, kTmemCols);
  pdl_wait();
  pdl_trigger();

  // ---- the shares of this pair's streams: a thread counts a run of requests
  if (blockIdx.x == 0 && tid == 0) check_offsets(p);
  if (rank == 0 && tid < 2) pieces.notes[2 * pair + tid].tokens = 0;
  const int run = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(p.B, tid * run), b_hi = min(p.B, b_lo + run);
  long long mine = 0, units;
  for (int b = b_lo; b < b_hi; ++b) mine += tree_units(p, load_request(p, b, blockIdx.x == 0), nodes);
  const long long before = scan_before<kWarps>(mine, sm.scan[0], units);
  const int used = (int)min((long long)kStreams, units);
  auto stream_of = [&](int t) { return 2 * pair + t; };
  auto begin_of = [&](int t) { return stream_of(t) < used ? share_begin(units, used, stream_of(t)) : 0; };
  auto end_of = [&](int t) { return stream_of(t) < used ? share_begin(units, used, stream_of(t) + 1) : 0; };
  const long long starts[2] = {begin_of(0), begin_of(1)};
#pragma unroll
  for (int t = 0; t < 2; ++t)
    if (starts[t] >= before && starts[t] < before + mine) {
      long long unit = before;
      int b = b_lo;
      for (; b + 1 < b_hi; ++b) {
        const long long here = tree_units(p, load_request(p, b, false), nodes);
        if (starts[t] < unit + here) break;
        unit += here;
      }
      sm.first_request[t] = b;
      sm.first_unit[t] = unit;
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
    more_registers<kSoftmaxRegs>();
    // (a call in a wait would bound the registers that this role may take)
    auto wait_here = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait<true>(bar, parity));
      return ok;
    };
    const int t = warp >> 2, r = tid & (kM - 1);
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = lanes + t * kTile, o_col = lanes + kColO + t * D, p_col = s_col + 64;
    const float c = p.scale * kLog2E;
    const float2 c2 = make_float2(c, c);
    const int tok_in = r / p.G, g_in = r - tok_in * p.G;
    const uint32_t p_half = cluster_addr(&sm.p_half[t], 0), p_full = cluster_addr(&sm.p_full[t], 0);
    int task = 0;
    Part part;
    for (int item = 0;; leave_part(t, item), ++item) {
      if (!wait_here(&sm.part_full[t][item % kNotes], (item / kNotes) & 1)) break;
      part = sm.part[t][item % kNotes];
      if (part.count == 0) break;
      const int L = part.L, n = part.n, token = part.token0 + rank * per_cta + tok_in;
      const bool live = tok_in < per_cta && token < n;
      const bool idle = !__any_sync(0xffffffffu, live);  // (what is left in P stays in rows that nobody reads)
      const int row_hi = live && L - n + token >= 0 ? L : 0;
      const int32_t* words = p.tree + (size_t)(part.t0 + min(token, n - 1)) * p.tree_words;
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      bool rounds = false;  // a maximum of the warp's is past kRounds
      for (int i = 0; i < part.count; ++i, ++task) {
        if (!wait_here(&sm.s_full[t][task % kRing], (task / kRing) & 1)) break;
        if (idle) {
          if (lane == 0) {
            mbar_arrive_cluster(p_half);
            mbar_arrive_cluster(p_full);
          }
          continue;
        }
        tc_fence_after();
        const int start = (part.tile0 + i) * kTile;
        // whole key tiles of a bf16 cache take x = c S in one product with the subtraction
        const bool whole = start + kTile <= L - n;
        const bool plain = !kE4m3 && whole && c >= 0.f;
        const float* scale = sm.slot[t].scale[kE4m3 ? task % kScales : 0][0];
        const float* v_scale = sm.slot[t].scale[kE4m3 ? task % kScales : 0][1];
        float x[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_32cols(s_col + 32 * q, x[q]);
        tmem_ld_wait();
        auto seen = [&](int at) {  // of the 32 positions from `at` on, by this row
          const uint32_t see = columns(0, row_hi - at);
          return row_hi > 0 ? see & tree_bits(words, p.tree_words, n, at - (L - n)) : see;
        };
        // Scores in units of log 2; what is not seen: -infinity.
        auto scored = [&](float(&y)[32], int col) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float2 a = c2, b = c2;
            if constexpr (kE4m3) {
              const float4 f = *reinterpret_cast<const float4*>(scale + col + e);
              a = make_float2(f.x, f.y);
              b = make_float2(f.z, f.w);
            }
            a = __fmul2_rn(make_float2(y[e], y[e + 1]), a);
            b = __fmul2_rn(make_float2(y[e + 2], y[e + 3]), b);
            y[e] = a.x;
            y[e + 1] = a.y;
            y[e + 2] = b.x;
            y[e + 3] = b.y;
          }
          if (!whole) {
            const int at = start + col;
            const uint32_t see = seen(at);
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
            float2 va = make_float2(exp2_approx(ya.x), exp2_approx(ya.y));
            float2 vb = make_float2(exp2_approx(yb.x), exp2_approx(yb.y));
            sum0 = __fadd2_rn(sum0, va);
            sum1 = __fadd2_rn(sum1, vb);
            if constexpr (kE4m3) {
              const float4 f = *reinterpret_cast<const float4*>(v_scale + 32 * q + e);
              va = __fmul2_rn(va, make_float2(f.x, f.y));
              vb = __fmul2_rn(vb, make_float2(f.z, f.w));
            }
            pw[e / 2] = pack_bf16(va.x, va.y);
            pw[e / 2 + 1] = pack_bf16(vb.x, vb.y);
          }
          if (kE4m3 && !whole) {  // 0 times a scale that is not finite
            const uint32_t see = seen(start + 32 * q);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pw[e] &= ((see >> 2 * e) & 1 ? 0x0000ffffu : 0u) | ((see >> 2 * e) & 2 ? 0xffff0000u : 0u);
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
      if (!ok || !wait_here(&sm.o_done[t][(task - 1) % kRing], ((task - 1) / kRing) & 1)) break;
      // ---- the end of this stream's part of the item
      tc_fence_after();
      const float l = l2.x + l2.y;
      const bool done = (part.flags & (kBegins | kEnds)) == (kBegins | kEnds);
      const int out_row = (part.t0 + token) * p.H + part.h * p.G + g_in;
      const size_t piece = ((size_t)stream_of(t) * 2 + (part.flags & kBegins ? 1 : 0)) * kRows + rank * kM + r;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool bad = !kE4m3 && sm.bad[t][item % kNotes] == item + 1;
      if (live) {
        if (!done) pieces.ml[piece] = make_float2(m, l);
        else if (p.lse) p.lse[out_row] = (m + log2f(l)) * kLn2;
      }
      if (rank == 0 && r == 0 && (part.flags & (kBegins | kEnds)) == kBegins)
        pieces.notes[stream_of(t)] = PieceNote{(part.t0 + part.token0) * p.H + part.h * p.G, min(nodes, n - part.token0),
                                               part.pieces, 0};
      int to_rows[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) to_rows[e] = __shfl_sync(0xffffffffu, live ? out_row : -1, (lane & ~3) + e);
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 32) {
        float o[32];
        tmem_ld_32cols(o_col + cc, o);
        tmem_ld_wait();
        if (!kE4m3 && bad && live) {
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = o[e];
          add_bad_nodes(p, part.b, part.h, L, n, max(part.tile0, max(0, L - n) / kTile) * kTile,
                               min(row_hi, (part.tile0 + part.count) * kTile), words,
                               p.q + (part.t0 + token) * p.q_stride + (size_t)(part.h * p.G + g_in) * D,
                               m == -INFINITY ? 0.f : m, cc, y);
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
    fewer_registers<kOtherRegs>();
    if (warp == kCopyWarp || warp == kCopyWarp + 1) {
      // ---- a stream's items: their notes, queries, keys and values.  (No division in the tiles' chain.)
      const int t = warp - kCopyWarp;
      Slot<kE4m3>& slot = sm.slot[t];
      const long long u0 = starts[t], u1 = end_of(t);
      const uint32_t key_ready = cluster_addr(sm.key_ready[t], 0), q_ready = cluster_addr(&sm.q_ready[t], 0);
      const int page_shift = 31 - __clz(p.c.page_size), in_page = p.c.page_size - 1;
      const int rows_per_box = min(p.c.page_size, kTile / 2), box_shift = min(page_shift, 6);
      const int half_boxes = (kTile / 2) >> box_shift, boxes = 2 * half_boxes;  // of a half, of a key tile
      const int nowhere = (p.c.num_pages * p.c.HKV) << page_shift;               // a row past the end: zeros
      int tasks = 0, item = 0;
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
      int b = 0, h = 0, tile = 0, tiles = 0;
      Request r{0, 0, 0};
      auto take = [&]() {  // the first request from b on that has nodes
        while (b < p.B) {
          r = load_request(p, b, false);
          if (r.n > 0) break;
          // (32 at a time: a million one by one would take longer than the others wait for a note)
          const unsigned some = __ballot_sync(0xffffffffu, b + lane < p.B && load_request(p, b + lane, false).n > 0);
          b += some ? __ffs(some) - 1 : 32;
        }
        h = tile = 0;
        tiles = (r.n + nodes - 1) / nodes;
      };
      if (u1 > u0) {
        b = sm.first_request[t];
        unit = sm.first_unit[t];
        take();
        const long long each = kItemCost + key_tiles(r.L), before = (u0 - unit) / each;  // items before u0's
        unit += before * each;
        h = (int)(before / tiles);
        tile = (int)(before - (long long)h * tiles);
      }
      while (u1 > u0 && unit < u1 && b < p.B && ok) {
        const int all = key_tiles(r.L);
        const int from = (int)max(0ll, u0 - unit - kItemCost), to = (int)min((long long)all, u1 - unit - kItemCost);
        if (to > from) {
          Part part;
          part.b = b;
          part.t0 = r.t0;
          part.n = r.n;
          part.L = r.L;
          part.h = h;
          part.token0 = tile * nodes;
          part.tile0 = from;
          part.count = to - from;
          part.flags = (from == 0 ? kBegins : 0) | (to == all ? kEnds : 0);
          part.pieces = to == all ? 1 : share_of(units, used, unit + kItemCost + all - 1) - stream_of(t) + 1;
          put_note(part);
          if (item > 0) wait(&sm.q_empty[t], (item - 1) & 1);
          ++item;
          if (!ok) break;
          if (rank == 0 && lane == 0) mbar_expect_tx(&sm.q_ready[t], 2 * kPanels * per_cta * p.G * 128);
          __syncwarp();
          if (lane < kPanels)
            tma_load_3d_pair(slot.q[lane], &q_map, q_ready, lane * 64, h * p.G, r.t0 + part.token0 + rank * per_cta);
          const int32_t* table = p.c.page_table + (size_t)b * p.c.max_pages;
          const int first = from * kTile, last = min(r.L, to * kTile);
          int page = -1;  // of the 32 boxes under way, by lane
          for (int i = 0; i < part.count; ++i, ++tasks) {
            if (((i * boxes) & 31) == 0) {
              const int pos = first + ((i * boxes + lane) << box_shift);
              page = -1;
              if (pos < last) {
                page = fresh(table + (pos >> page_shift));
                if (page < 0 || page >= p.c.num_pages) {
                  raise_status(p.dev_status, KDA_DEV_BAD_PAGE);
                  page = -1;
                }
              }
            }
            // rows of the cache where the tile's boxes start, by lane; past the end: zeros
            const int box = lane & (boxes - 1), at = i * boxes + box;
            const int pg = __shfl_sync(0xffffffffu, page, at & 31);
            const int row = pg >= 0 ? ((pg * p.c.HKV + h) << page_shift) + ((first + (at << box_shift)) & in_page) : nowhere;
            const int s = tasks % kRing, before = tasks / kRing - 1;  // what was there before: key tile tasks - kRing
            if constexpr (!kE4m3) {
              // this CTA's half of the keys; both CTAs' copies arrive at the first's barrier
              const int half_row = __shfl_sync(0xffffffffu, row, rank * half_boxes + (lane & (half_boxes - 1)));
              const int panel = lane / half_boxes;
              if (before >= 0) wait(&sm.s_full[t][s], before & 1);
              if (!ok) break;
              if (rank == 0 && lane == 0) mbar_expect_tx(&sm.key_ready[t][s], 2 * kKeyBytes);
              __syncwarp();
              if (panel < kPanels)
                tma_load_3d_pair(slot.key[s] + panel * kKeyPanel + (lane & (half_boxes - 1)) * rows_per_box * 128, &k_map,
                                 key_ready + 8 * s, 0, half_row, panel);
              // its columns of all values
              if (before >= 0) wait(&sm.o_done[t][s], before & 1);
              if (!ok) break;
              if (lane == 0) mbar_expect_tx(&sm.value_full[t][s], kValueBytes);
              __syncwarp();
              if (lane < boxes)
                tma_load_3d(slot.value[s] + lane * rows_per_box * 128, &v_map, &sm.value_full[t][s], 0, row, rank);
            } else {
              // codes of this CTA's half of the keys, and all scales; codes of its columns of all values.
              // Scales of positions without a page are zeros.
              const unsigned real = __ballot_sync(0xffffffffu, lane < boxes && pg >= 0);
              const uint32_t scale_bytes = __popc(real) * rows_per_box * 4;
              float* scale = slot.scale[tasks % kScales][0] + lane * rows_per_box;
              if (before >= 0) wait(&sm.key_free[t][s], before & 1);
              if (!ok) break;
              if (lane < boxes && pg < 0) {
                for (int e = 0; e < rows_per_box; ++e) scale[e] = scale[kTile + e] = 0.f;
                fence_proxy_async_smem();
              }
              __syncwarp();
              if (lane == 0) mbar_expect_tx(&sm.key_full[t][s], kRawBytes + 2 * scale_bytes);
              __syncwarp();
              if (lane < boxes) {
                if (lane / half_boxes == rank)
                  tma_load_2d(slot.raw_key[s] + (lane & (half_boxes - 1)) * rows_per_box * D, &k_map,
                              &sm.key_full[t][s], 0, row);
                if (pg >= 0) {
                  bulk_load(scale, p.c.k_scale + row, rows_per_box * 4, &sm.key_full[t][s]);
                  bulk_load(scale + kTile, p.c.v_scale + row, rows_per_box * 4, &sm.key_full[t][s]);
                }
              }
              if (before >= 0) wait(&sm.value_free[t][s], before & 1);
              if (!ok) break;
              if (lane == 0) mbar_expect_tx(&sm.value_full[t][s], kRawBytes);
              __syncwarp();
              if (lane < boxes)
                tma_load_2d(slot.raw_value[s] + lane * rows_per_box * (D / 2), &v_map, &sm.value_full[t][s],
                            rank * (D / 2), row);
            }
          }
        }
        unit += kItemCost + all;
        if (++tile >= tiles) {
          tile = 0;
          if (++h >= p.c.HKV) {
            ++b;
            take();
          }
        }
      }
      if (ok) put_note(Part{0, 0, 0, 0, 0, 0, 0, 0, 0, 0});
      if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
      // Every copy lands before the CTA's memory is released.  (Also when a wait gave up: then a second has
      // passed since the last copy that is not waited for here.)
      for (int u = max(0, tasks - kRing); u < tasks; ++u) {
        mbar_wait(&sm.value_full[t][u % kRing], (u / kRing) & 1);
        if (kE4m3) mbar_wait(&sm.key_full[t][u % kRing], (u / kRing) & 1);
        else if (rank == 0) mbar_wait(&sm.key_ready[t][u % kRing], (u / kRing) & 1);
      }
      if (rank == 0 && item > 0) mbar_wait(&sm.q_ready[t], (item - 1) & 1);
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
        const int s = here.tasks % kRing;
        if (!wait(&sm.key_ready[t][s], (here.tasks / kRing) & 1)) return;
        tc_fence_after();
        --here.left;
        const uint64_t a = smem_desc_sw128(smem_u32(sm.slot[t].q[0]), 16, 1024);
        const uint64_t k = smem_desc_sw128(smem_u32(sm.slot[t].key[kE4m3 ? 0 : s]), 16, 1024);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)  // 32 bytes on, or the next panel
          mma_bf16_pair_if(one, base + t * kTile, a + (j & 3) * 2 + (j >> 2) * (kQPanel / 16),
                           k + (j & 3) * 2 + (j >> 2) * (kKeyPanel / 16), idesc_s, j > 0 ? 1u : 0u);
        mma_commit_pair_if(one, &sm.s_full[t][s]);
        if (here.left == 0) mma_commit_pair_if(one, &sm.q_empty[t]);
        here.live = true;
      };
      auto output = [&](int t) {  // PV of the slot's S under way
        const int s = here.tasks % kRing;
        const uint32_t d = base + kColO + t * D, pc = base + t * kTile + 64;
        const uint64_t v = smem_desc_sw128(smem_u32(sm.slot[t].value[kE4m3 ? 0 : s]), kTile * 128, 1024);
        wait(&sm.value_ready[t][s], (here.tasks / kRing) & 1);
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
    } else if (warp >= kPrepareWarp) {
      // ---- codes to bf16, and values without the entries that some row must not see: two warps a slot
      const int t = (warp - kPrepareWarp) >> 1, at = tid & 63;
      Slot<kE4m3>& slot = sm.slot[t];
      const uint32_t key_ready = cluster_addr(sm.key_ready[t], 0), value_ready = cluster_addr(sm.value_ready[t], 0);
      int tasks = 0;
      Part part;
      for (int item = 0; read_part(t, item, part); leave_part(t, item), ++item) {
        for (int i = 0; i < part.count; ++i, ++tasks) {
          const int s = tasks % kRing, start = (part.tile0 + i) * kTile;
          const uint32_t phase = (tasks / kRing) & 1;
          const bool whole = start + kTile <= part.L - part.n;
          const int to = part.L - start;  // the request's keys
          bool bad = false;
          if constexpr (kE4m3) {
            if (!wait(&sm.key_full[t][s], phase)) break;
            float* scale = slot.scale[tasks % kScales][0];
            scale[at] *= p.scale * kLog2E;
            scale[at + 64] *= p.scale * kLog2E;
            if (tasks > 0 && !wait(&sm.s_full[t][(tasks - 1) % kRing], ((tasks - 1) / kRing) & 1)) break;
#pragma unroll 4
            for (int e = 0; e < 8; ++e) {  // 16 codes of a key: eight lanes write two keys' chunks, in different banks
              const int n = e * 64 + at, key = (n >> 4) * 2 + ((n >> 2) & 1), ch = (n & 3) + ((n >> 3) & 1) * 4;
              const uint4 x = *reinterpret_cast<const uint4*>(slot.raw_key[s] + key * D + ch * 16);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
              uint32_t y[8];
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                y[2 * d] = widen(__byte_perm(w[d], 0, 0x1404));
                y[2 * d + 1] = widen(__byte_perm(w[d], 0, 0x3424));
              }
              unsigned char* panel = slot.key[0] + (ch >> 2) * kKeyPanel;
              *reinterpret_cast<uint4*>(panel + swizzled<128>(key, (2 * ch) & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(panel + swizzled<128>(key, (2 * ch + 1) & 7)) =
                  make_uint4(y[4], y[5], y[6], y[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&sm.key_free[t][s]);
              mbar_arrive_cluster(key_ready + 8 * s);
            }
            if (!wait(&sm.value_full[t][s], phase)) break;
            if (tasks > 0 && !wait(&sm.o_done[t][(tasks - 1) % kRing], ((tasks - 1) / kRing) & 1)) break;
#pragma unroll 2
            for (int e = 0; e < 8; ++e) {
              const int n = e * 64 + at, key = n >> 2, ch = n & 3;
              const uint4 x = *reinterpret_cast<const uint4*>(slot.raw_value[s] + key * (D / 2) + ch * 16);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
              uint32_t y[8];
#pragma unroll
              for (int d = 0; d < 8; ++d) y[d] = widen(__byte_perm(w[d >> 1], 0, d & 1 ? 0x3424 : 0x1404));
              *reinterpret_cast<uint4*>(slot.value[0] + swizzled<128>(key, 2 * ch)) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(slot.value[0] + swizzled<128>(key, 2 * ch + 1)) =
                  make_uint4(y[4], y[5], y[6], y[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.value_free[t][s]);
          } else {
            if (!wait(&sm.value_full[t][s], phase)) break;
            if (!whole) {
#pragma unroll 4
              for (int e = 0; e < kTile * 8 / 64; ++e) {
                const int n = e * 64 + at, key = n >> 3;
                uint4* x = reinterpret_cast<uint4*>(slot.value[s] + swizzled<128>(key, n & 7));
                const uint4 y = *x;
                const uint4 out = make_uint4(not_finite(y.x), not_finite(y.y), not_finite(y.z), not_finite(y.w));
                const bool some = (out.x | out.y | out.z | out.w) != 0;
                bad |= key < to && some;
                if (key >= to) *x = make_uint4(0, 0, 0, 0);
                else if (some) *x = make_uint4(y.x & ~out.x, y.y & ~out.y, y.z & ~out.z, y.w & ~out.w);
              }
              fence_proxy_async_smem();
            }
          }
          if (__any_sync(0xffffffffu, bad)) {  // the rows of either CTA add them at the item's end
            if (lane == 0)
              for (int to = 0; to < 2; ++to)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&sm.bad[t][item % kNotes], to)),
                             "r"(item + 1)
                             : "memory");
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(value_ready + 8 * s);
        }
        if (!ok) break;
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
// CTA (c, y) takes 16 columns from 16 (y / 2) on of the rows of CTA y % 2 in the item that stream c began.
constexpr int kJoinY = 2 * D / 16;
__global__ void __launch_bounds__(kM) tree_join_kernel(const AttentionArgs p, const Pieces s) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, cc = blockIdx.y >> 1, rank = blockIdx.y & 1, row = rank * kM + threadIdx.x;
  const PieceNote note = s.notes[c];
  const int per_cta = kM / p.G, tok_in = threadIdx.x / p.G, token = rank * per_cta + tok_in;
  if (tok_in >= per_cta || token >= note.tokens) return;
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
  const size_t out_row = (size_t)note.row0 + (size_t)token * p.H + (threadIdx.x - tok_in * p.G);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint4* to = reinterpret_cast<uint4*>(p.out + out_row * D + 16 * cc);
#pragma unroll
  for (int e = 0; e < 4; e += 2)
    to[e / 2] = make_uint4(pack_bf16(o[e].x * inv, o[e].y * inv), pack_bf16(o[e].z * inv, o[e].w * inv),
                           pack_bf16(o[e + 1].x * inv, o[e + 1].y * inv), pack_bf16(o[e + 1].z * inv, o[e + 1].w * inv));
  if (p.lse && cc == 0) p.lse[out_row] = (m + log2f(l)) * kLn2;
}

template <bool kE4m3>
cudaError_t launch_tree(const AttentionArgs& a, cudaStream_t stream) {
  static_assert(sizeof(TreeSmem<kE4m3>) + 1024 <= 227 * 1024, "a CTA fits an SM");
  CUtensorMap q_map, maps[2];
  if (!make_map_3d_bf16(&q_map, a.q, D, a.H, a.T, D * 2, (uint64_t)a.q_stride * 2, 64, a.G, kM / a.G))
    return cudaErrorInvalidValue;
  const uint64_t rows = (uint64_t)a.c.num_pages * a.c.HKV * a.c.page_size;
  const uint32_t rows_per_box = a.c.page_size < kTile / 2 ? a.c.page_size : kTile / 2;
  for (int i = 0; i < 2; ++i) {
    const void* cache = i ? a.c.v : a.c.k;
    // bf16: the cache as [panel of 64 entries][row][64 entries]
    const bool made = kE4m3 ? make_map_2d(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, cache, D, rows, i ? D / 2 : D,
                                          rows_per_box, CU_TENSOR_MAP_SWIZZLE_NONE)
                            : make_map_3d_bf16(&maps[i], cache, 64, rows, kPanels, D * 2, 128, 64, rows_per_box, 1);
    if (!made) return cudaErrorInvalidValue;
  }
  const size_t smem = sizeof(TreeSmem<kE4m3>) + 1024;
  static SmemSet set;
  cudaError_t e = allow_smem(tree_kernel<kE4m3>, smem, set);
  if (e != cudaSuccess) return e;
  const Pieces pieces = pieces_at(a.workspace, kStreams, kRows);
  e = launch_pairs(tree_kernel<kE4m3>, dim3(2 * kPairs), dim3(kThreads), smem, stream, q_map, maps[0], maps[1], a, pieces);
  if (e != cudaSuccess) return e;
  return launch(tree_join_kernel, dim3(kStreams, kJoinY), dim3(kM), 0, stream, true, a, pieces);
}

}  // namespace

size_t tree_pairs_bytes() { return (pieces_bytes(kStreams, kRows, D) + 255) & ~(size_t)255; }

cudaError_t launch_tree_pairs(const AttentionArgs& a, cudaStream_t stream) {
  return a.c.e4m3 ? launch_tree<true>(a, stream) : launch_tree<false>(a, stream);
}

}  // namespace kda
