// kda_attn_chunk.cuh -- attention of chunks: the requests with more rows (new tokens x
// query heads per key head) than the window kernel takes, and drafted trees over heads of 64 (kTree).
//
// Such a request does 4 D operations per row and cached position on 4 D bytes per
// position: with hundreds of rows the tensor cores bound it.  One CTA per SM
// works on items of one or two row tiles of 128 (row i G + g: token i, head g of the
// group) of one (request, key head), and key tiles of 128 positions.  A task is a
// (row tile, key tile):
//   S = Q K^T        128 x 128, TMEM; K-major operands from shared memory
//   P = 2^(S - m)    in bf16, back to TMEM by the 128 threads that own one row each
//   O += P V         TMEM; A = P from TMEM, B = V from shared memory (N-major)
// Tasks take two slots (S, P, O and four softmax warps each) in turn: while one
// slot's softmax runs, the other's products do.  An item of two row tiles has one in
// each slot; an item of one row tile deals its key tiles to both, and their two
// outputs are joined at its end.  A warp per slot issues its products, PV of task k
// and then S of task k + 2, and runs on into the next item; the two warps take
// turns, since products of both slots mixed would end together, and then both
// slots' softmax would run at once and the tensor cores wait.  For D = 128, a slot's
// S and P share columns: the tensor cores take one thread's products in order, so
// the next S starts when PV has read P.  P is handed over in halves.
// O is rescaled only when a row's maximum has grown by more than 2^8: weights up to
// 256 lose nothing in bf16, and after the first key tiles that hardly ever happens.
//
// K and V come through TMA, one box per page and 128-byte panel.  An e4m3 cache's
// codes are widened to bf16 by four more warps on the way; a key's scale
// multiplies its column of S, a value's scale its column of P.
//
// Items' key tiles are divided evenly over the CTAs, an item's ends counted as some.
//
// 2048 new tokens over 28001 cached, 32 / 8 heads, D = 128, bf16: 638 us alone, 1.53 PFLOP/s,
// 706 among other calls, 1.38 (a cuBLAS product: 1.89), the tensor cores busy for two thirds;
// a softmax task is a chain of some 3000 cycles beside the 1280 of its products, and two of
// them overlap.  Four prompts of 1500 .. 6001 from an e4m3 cache: 727 us, 0.68 PFLOP/s: the scales are a
// product and the widening five operations per pair, and the schedulers issue in 54% of their cycles.
// (e4m3 operands widened to f16 as in the window kernel: 1149 us against 818 then, the
// conversions run where the exponentials do.  Codes taken to registers one part ahead:
// 882 against 847.)
//
// A key tile that some row sees in part (the diagonal, the window's edge, the
// sequence's end, a tree) is masked in the softmax, and entries of V that are outside the
// request's range, or not finite, are taken out of shared memory first (0 x NaN
// would reach the rows that do not see them); an item that had live entries of
// that kind adds them, for the rows that see them, at its end.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "kda_attn.cuh"
#include "kda_launch.h"
#include "kda_tcgen05.cuh"
#include "kda_tmap.h"

namespace kda {
namespace {

constexpr int kTile = 128;          // positions per key tile
constexpr int kM = 128;             // rows per row tile
// Warps: 0-3 and 4-7 the slots' softmax, 8 and 9 their products, then one each for
// what is copied and for V's entries that are not finite; for e4m3 four more that
// widen the codes.
constexpr int kMmaWarp = 8, kCopyWarp = 10, kWidenWarp = 12;
constexpr int kSteps = 8;           // steps whose notes and barriers are kept: more than the rings hold
constexpr float kGrow = 8.f;        // growth of a maximum (log 2) that rescales O
constexpr float kRounds = 4194304.f;  // maxima past 2^22: half an fp32 step is more than 2^-2

// What the product and the fixing warps need to know of a step (one key tile of
// one item); the copying warp for K and V writes it before K.
struct StepNote {
  int flags;
  int start;             // first position of the key tile
  int begin, end;        // positions of the request that any of its tokens sees
  int item;              // running number in this CTA
  int index;             // of the step in this CTA's part of the item
};
constexpr int kFirst = 1, kLast = 2;  // of this CTA's part of the item
constexpr int kSecond = 8;            // the item has a second row tile
constexpr int kWhole = 16;            // every row sees every position

// Where a unit of work is: its item, the key tile (0 where the unit stands for none), the item's
// first unit, and how many units before it stand for no key tile.
struct Place {
  int b, h, token0, tile;
  long long item_unit, idle;
};

template <int D, bool kE4m3, bool kPair>
struct Shape {
  static constexpr int kPanels = D / 64;
  static constexpr int kUnitBytes = kTile * D * 2;       // K or V of one key tile, bf16
  static constexpr int kQTiles = kPair ? 2 : 1;
  // units alternate K, V, K, V ..; four are the least that S two tasks ahead needs, and as
  // many as fit are taken: with a key tile per task (kPair false) copies have to be far ahead
  static constexpr int kUnits = D == 128 ? (kE4m3 ? 4 : 5) + (kPair ? 0 : 1) : kE4m3 ? 8 : 12;
  static constexpr int kPart = kE4m3 ? 64 : 128;         // positions copied at a time
  static constexpr int kRawUnits = kE4m3 ? (D == 128 ? 3 : 6) : 1;  // parts of codes
  static constexpr int kRawBytes = kPart * D;
  static constexpr int kScaleSteps = D == 128 ? 4 : 8;   // steps whose scales are kept
  // What an item's beginning and end take, in key tiles, so that shares with many short items
  // end with the others.  1, 2, 3, 4 tiles: six prompts of 300 .. 4000 in bf16 272, 255, 249,
  // 245 us; 0, 1, 2, 3: four of 1500 .. 6001 in e4m3 820, 762, 732, 742 us.
  static constexpr int kItemCost = kE4m3 ? 2 : 4;
  static constexpr int kWarps = kE4m3 ? 16 : 12;
  static constexpr int kThreads = 32 * kWarps;
  // Registers per thread: 65536 (e4m3) or 64512 at launch, then dealt by role to no more
  static constexpr int kSoftmaxRegs = kE4m3 ? 152 : 208;
  static constexpr int kOtherRegs = kE4m3 ? 72 : 88;
  [[maybe_unused]] static constexpr int kWidenRegs = 120;
  static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs + (kE4m3 ? 128 * kWidenRegs : 0) <=
                    kThreads * (65536 / kThreads & ~7),
                "the roles' registers fit in the launch's");
  // TMEM: S of both slots in columns 0 .. 255, O of both from kColO on; P in the second
  // half of its S (D = 128, where S and PV have one shape and so complete in the order
  // of issue), or in columns of its own
  static constexpr uint32_t kColO = 256;
  __host__ __device__ static constexpr uint32_t col_p(int t) { return D == 128 ? t * kTile + 64 : 384 + 64 * t; }
};
constexpr uint32_t kTmemCols = 512;

template <int D, bool kE4m3, bool kPair>
struct Smem {
  using S = Shape<D, kE4m3, kPair>;
  unsigned char q[S::kQTiles][kM * D * 2];         // 1024-aligned, swizzled panels
  unsigned char unit[S::kUnits][S::kUnitBytes];
  unsigned char raw[kE4m3 ? S::kRawUnits : 1][kE4m3 ? S::kRawBytes : 16];
  float raw_scale[kE4m3 ? S::kRawUnits : 1][kE4m3 ? S::kPart : 4];
  float scale[kE4m3 ? S::kScaleSteps : 1][2][kE4m3 ? kTile : 4];  // by step: K's (times the score scale), V's
  float2 other[kM];                                // the second slot's maxima and sums, to be joined
  float2 rows[kE4m3 ? 2 : 1][kE4m3 ? kM : 1];     // maxima and sums on their way between layouts
  StepNote note[kSteps];
  int bad[kSteps];                                 // by item: live entries of V were taken out
  uint64_t full[S::kUnits], empty[S::kUnits], fixed[kSteps];
  uint64_t raw_full[S::kRawUnits], raw_empty[S::kRawUnits];
  uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_done[2], turn[2], done, join_ready, join_done;
  long long part[2][S::kWarps];
  Place edge[2];          // of the first unit of this CTA, of the first one past it
  uint32_t tmem;
};

// The item's key tiles: from tile `first`, `tiles` of them (at least one: rows that
// see nothing are written too).
struct Span {
  int first, tiles;
};
__device__ __forceinline__ Span span_of(const AttentionArgs& p, const Request& r, int token0, int tokens) {
  const int pos0 = r.L - r.n;
  const int last = pos0 + min(r.n, token0 + tokens) - 1;
  const int lo = seen_lo(p, max(0, pos0 + token0)), hi = min(seen_hi(p, last, r.L), r.L);
  const int first = lo / kTile;
  return Span{first, max(1, (hi + kTile - 1) / kTile - first)};
}
// Units of one key head of a request (0: not this kernel's), `pair` tokens to an item: an
// item's are `cost` for its beginning and end, then one per key tile.
__device__ __forceinline__ int head_items(const AttentionArgs& p, const Request& r, int pair) {
  return r.n * p.G <= p.window_rows ? 0 : (r.n + pair - 1) / pair;
}
__device__ __forceinline__ long long head_units(const AttentionArgs& p, const Request& r, int pair, int cost) {
  if (r.n * p.G <= p.window_rows) return 0;
  long long sum = 0;
  for (int t = 0; t < r.n; t += pair) sum += span_of(p, r, t, pair).tiles + cost;
  return sum;
}
// The place of unit u in request at.b, whose first unit is at.item_unit, with at.idle items
// before it; by a whole warp.
__device__ __forceinline__ Place place_of(const AttentionArgs& p, Place at, long long u, int pair, int cost, int lane) {
  const Request r = load_request(p, at.b, false);
  const int items = head_items(p, r, pair);
  auto units_of = [&](int i) { return i < items ? span_of(p, r, i * pair, pair).tiles + cost : 0; };
  long long head = 0;
  for (int i = lane; i < items; i += 32) head += units_of(i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) head += __shfl_xor_sync(0xffffffffu, head, o);
  at.h = (int)((u - at.item_unit) / head);
  long long left = u - at.item_unit - at.h * head;  // less than the head's units
  int first = 0;
  while (true) {
    const int mine = units_of(first + lane);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, left < upto);
    if (past || first + 32 >= items) {
      const int in = past ? __ffs(past) - 1 : 0;
      left -= __shfl_sync(0xffffffffu, upto - mine, in);
      first += in;
      break;
    }
    left -= __shfl_sync(0xffffffffu, upto, 31);
    first += 32;
  }
  at.token0 = first * pair;
  at.tile = max(0, (int)left - cost);
  at.item_unit = u - left;
  at.idle = (at.idle + (long long)at.h * items + first) * cost + min(left, (long long)cost);
  return at;
}

// The items of one CTA's share in order (request, key head, row tiles), walked by a
// whole warp: 32 requests are looked up at a time.
struct Walk {
  int base;
  Request mine;
  int b, h, token0;
  Request r;
  Span span;
  int tile;         // next key tile of the item, 0 .. span.tiles - 1
  long long left;

  __device__ __forceinline__ void fetch(const AttentionArgs& p, int lane) {
    base = b;
    mine = Request{0, 0, 0};
    if (b + lane < p.B) mine = load_request(p, b + lane, false);
    if (mine.n * p.G <= p.window_rows) mine.n = 0;
  }
  __device__ __forceinline__ void take(const AttentionArgs& p, int pair, int lane) {
    while (b < p.B) {
      if (b >= base + 32) fetch(p, lane);
      const unsigned some = __ballot_sync(0xffffffffu, mine.n > 0) & (0xffffffffu << (b - base));
      if (some) {
        const int src = __ffs(some) - 1;
        b = base + src;
        r.t0 = __shfl_sync(0xffffffffu, mine.t0, src);
        r.n = __shfl_sync(0xffffffffu, mine.n, src);
        r.L = __shfl_sync(0xffffffffu, mine.L, src);
        token0 = 0;
        span = span_of(p, r, 0, pair);
        return;
      }
      b = base + 32;
    }
    left = 0;  // cannot happen while units are left
  }
  __device__ __forceinline__ void start(const AttentionArgs& p, int pair, const Place& at, long long tiles, int lane) {
    b = at.b;
    left = tiles;
    fetch(p, lane);
    take(p, pair, lane);
    h = at.h;
    token0 = at.token0;
    span = span_of(p, r, token0, pair);
    tile = at.tile;
  }
  __device__ __forceinline__ int count() const { return (int)min((long long)(span.tiles - tile), left); }
  __device__ __forceinline__ void next(const AttentionArgs& p, int pair, int lane) {
    left -= count();
    if (left <= 0) return;
    tile = 0;
    token0 += pair;
    if (token0 >= r.n) {
      token0 = 0;
      if (++h == p.c.HKV) {
        h = 0;
        ++b;
        take(p, pair, lane);
        return;
      }
    }
    span = span_of(p, r, token0, pair);
  }
};

// All steps of 16 along the contraction of S = Q K^T.  `turn` goes to the other slot's
// warp before the last two: what is queued by then covers its waking up.  (The loop is
// unrolled twice only: the softmax's code leaves little of the instruction cache to
// this; all eight steps in line took 753 us where this takes 731.)
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t q_addr, uint32_t k_addr, uint64_t* turn) {
  const uint32_t idesc = idesc_bf16(kTile, kM, false, false);
  uint64_t a = smem_desc_sw128(q_addr, 16, 1024), b = smem_desc_sw128(k_addr, 16, 1024);
#pragma unroll 2
  for (int j = 0; j < D / 16; ++j) {
    if (j == D / 16 - 2 && turn) mbar_arrive(turn);
    mma_bf16(d, a, b, idesc, j > 0 ? 1u : 0u);
    const uint32_t step = (j & 3) == 3 ? kM * 128 / 16 - 6 : 2;  // 32 bytes on, or the next panel
    a += step;
    b += step;
  }
}
// The steps of O (+)= P V over one half of the key tile.
template <int D, int kHalf>
__device__ __forceinline__ void issue_output(uint32_t d, uint32_t p_col, uint32_t v_addr, bool add) {
  const uint32_t idesc = idesc_bf16(D, kM, false, true);
  const uint64_t b = smem_desc_sw128(v_addr, kTile * 128, 1024);
#pragma unroll
  for (int j = 4 * kHalf; j < 4 * kHalf + 4; ++j)
    mma_bf16_tmem_a(d, p_col + 8 * j, b + ((j * 16 * 128) >> 4), idesc, (add || j > 4 * kHalf) ? 1u : 0u);
}

// The halves of v (two bf16) that are not finite, as a mask.
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  return ((v & 0x7f80u) == 0x7f80u ? 0x0000ffffu : 0u) | ((v & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// Whether rows with positions first .. last all see every position of the key tile; n: the
// request's new tokens, a tree of which is seen in part.
template <bool kTree>
__device__ __forceinline__ bool sees_whole(const AttentionArgs& p, int L, int n, int first, int last, int start) {
  if (kTree) return start + kTile <= L - n;
  return start >= seen_lo(p, last) && start + kTile <= min(seen_hi(p, first, L), L);
}

// Adds the live entries of V that were taken out of an item's partly seen key tiles
// (`steps` of them from position start0 on; its rows are at positions first .. last)
// to columns col .. col + 31 of one row's output: the weight of each is found
// again from Q and K in memory.  (Rare: values that are not finite.)
template <int D, bool kTree>
__device__ __noinline__ void add_bad_values(const AttentionArgs& p, int b, int h, int L, int n, int pos, int first,
                                            int last, int start0, int steps, const int32_t* words, const kda_bf16* q,
                                            float m, int col, float* o) {
  const int lo = seen_lo(p, pos), hi = min(seen_hi(p, pos, L), L);
  const kda_bf16* kc = static_cast<const kda_bf16*>(p.c.k);
  const kda_bf16* vc = static_cast<const kda_bf16*>(p.c.v);
  const int32_t* table = p.c.page_table + (size_t)b * p.c.max_pages;
  for (int s = 0; s < steps; ++s) {
    const int start = start0 + s * kTile;
    if (sees_whole<kTree>(p, L, n, first, last, start)) continue;
    for (int j = max(lo, start); j < min(hi, start + kTile); ++j) {
      if (kTree && !(tree_bits(words, p.tree_words, n, j - (L - n)) & 1)) continue;
      const int page = table[j / p.c.page_size];
      if (page < 0 || page >= p.c.num_pages) continue;
      const size_t row = ((size_t)page * p.c.HKV + h) * p.c.page_size + j % p.c.page_size;
      float w = -1.f;
      for (int d = 0; d < 32; ++d) {
        const uint32_t v = vc[row * D + col + d];
        if ((v & 0x7f80u) != 0x7f80u) continue;
        if (w < 0.f) {
          float x = 0.f;
          for (int e = 0; e < D; ++e)
            x = fmaf(__uint_as_float((uint32_t)q[e] << 16), __uint_as_float((uint32_t)kc[row * D + e] << 16), x);
          w = exp2_approx(x * (p.scale * kLog2E) - m);
        }
        o[d] = fmaf(w, __uint_as_float(v << 16), o[d]);
      }
    }
  }
}

// kPair: items may have two row tiles (else no request of the call has more than one).
// kTree: the new tokens are a tree's, each of which sees those that its mask names.
template <int D, bool kE4m3, bool kPair, bool kTree>
__global__ void __launch_bounds__(Shape<D, kE4m3, kPair>::kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const AttentionArgs p, const Pieces pieces) {
  using S = Shape<D, kE4m3, kPair>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D, kE4m3, kPair>& sm = *reinterpret_cast<Smem<D, kE4m3, kPair>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int per_tile = kM / p.G;     // tokens of a row tile
  const int pair = 2 * per_tile;     // of an item

  if (tid == 0) {
    for (int s = 0; s < S::kUnits; ++s) {
      mbar_init(&sm.full[s], kE4m3 ? 4 : 1);
      mbar_init(&sm.empty[s], 2);
    }
    for (int s = 0; s < kSteps; ++s) mbar_init(&sm.fixed[s], 1);
    for (int s = 0; s < S::kRawUnits; ++s) {
      mbar_init(&sm.raw_full[s], 1);
      mbar_init(&sm.raw_empty[s], 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.q_full[t], 1);
      mbar_init(&sm.q_empty[t], 2);
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_half[t], 4);
      mbar_init(&sm.p_full[t], 4);
      mbar_init(&sm.o_done[t], 1);
      mbar_init(&sm.turn[t], 1);
    }
    mbar_init(&sm.join_ready, 4);
    mbar_init(&sm.join_done, 4);
    mbar_init(&sm.done, 2);
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem, kTmemCols);
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share: each thread counts a run of requests
  if (cta == 0 && tid == S::kThreads - 1) check_offsets(p);
  const int run = (p.B + S::kThreads - 1) / S::kThreads;
  const int b_lo = min(p.B, tid * run), b_hi = min(p.B, b_lo + run);
  long long mine = 0, my_items = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Request r = load_request(p, b, cta == 0);
    mine += p.c.HKV * head_units(p, r, pair, S::kItemCost);
    my_items += p.c.HKV * head_items(p, r, pair);
  }
  long long units, items;
  const long long from = scan_before<S::kWarps>(mine, sm.part[0], units);
  const long long items_from = scan_before<S::kWarps>(my_items, sm.part[1], items);
  const int used = (int)min((long long)ctas, units);
  if (tid == 0) pieces.notes[cta].tokens = 0;
  const long long u0 = cta < used ? share_begin(units, used, cta) : 0;
  const long long u1 = cta < used ? share_begin(units, used, cta + 1) : 0;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const long long u = i ? u1 : u0;
    if (u1 <= u0 || u < from || u >= from + mine) continue;
    Place at{b_lo, 0, 0, 0, from, items_from};
    for (; at.b + 1 < b_hi; ++at.b) {
      const Request r = load_request(p, at.b, false);
      const long long n = p.c.HKV * head_units(p, r, pair, S::kItemCost);
      if (u < at.item_unit + n) break;
      at.item_unit += n;
      at.idle += p.c.HKV * head_items(p, r, pair);
    }
    sm.edge[i] = at;
  }
  __syncthreads();
  if (warp < 2) {
    const long long u = warp ? u1 : u0;
    Place at{0, 0, 0, 0, 0, items * S::kItemCost};  // past the last unit
    if (u1 > u0 && u < units) at = place_of(p, sm.edge[warp], u, pair, S::kItemCost, lane);
    __syncwarp();
    if (lane == 0) sm.edge[warp] = at;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int steps = u1 > u0 ? (int)((u1 - sm.edge[1].idle) - (u0 - sm.edge[0].idle)) : 0;  // key tiles
  bool ok = true;

  if (warp >= kWidenWarp) {
    if constexpr (kE4m3) {
      // ---- codes to bf16, four warps
      fewer_registers<S::kWidenRegs>();
      const int at = tid - 32 * kWidenWarp;
      for (int r = 0; r < 4 * steps && ok; ++r) {  // parts: two of K, two of V
        const int u = r >> 1, s = u % S::kUnits, g = u >> 1, kv = u & 1, part = r & 1, rs = r % S::kRawUnits;
        ok = mbar_wait(&sm.raw_full[rs], (r / S::kRawUnits) & 1);
        if (part == 0 && u >= S::kUnits) ok = ok && mbar_wait(&sm.empty[s], (u / S::kUnits - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (at < S::kPart) {
          const float f = sm.raw_scale[rs][at];
          sm.scale[g % S::kScaleSteps][kv][part * S::kPart + at] = kv ? f : f * (p.scale * kLog2E);
        }
        constexpr int kPieces = D / 16;  // 16-code pieces of a row
        constexpr int kEach = S::kPart * kPieces / 128;
        // Eight lanes write two rows by four pieces, whose chunks lie in different banks.
        auto piece = [&](int i) {  // row, piece
          const int n = i * 128 + at;
          return kPieces == 8 ? make_int2((n >> 4) * 2 + ((n >> 2) & 1), (n & 3) + ((n >> 3) & 1) * 4)
                              : make_int2(n >> 2, n & 3);
        };
        uint4 x[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
          x[i] = *reinterpret_cast<const uint4*>(sm.raw[rs] + piece(i).x * D + piece(i).y * 16);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int to_row = part * S::kPart + piece(i).x, c = piece(i).y;
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[2 * e] = widen(__byte_perm(w[e], 0, 0x1404));
            y[2 * e + 1] = widen(__byte_perm(w[e], 0, 0x3424));
          }
          unsigned char* to = sm.unit[s] + ((2 * c) >> 3) * kTile * 128;
          *reinterpret_cast<uint4*>(to + swizzled<128>(to_row, (2 * c) & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(to + swizzled<128>(to_row, (2 * c + 1) & 7)) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.raw_empty[rs]);
          if (part == 1) mbar_arrive(&sm.full[s]);
        }
      }
      if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
    }
  } else if (warp >= kMmaWarp) {
    fewer_registers<S::kOtherRegs>();
    if (steps == 0) {
      // nothing to do
    } else if (warp == kCopyWarp) {
      // ---- notes, the items' queries, and K and V of every step into the ring
      Walk w;
      w.start(p, pair, sm.edge[0], steps, lane);
      const int rows_per_box = min(p.c.page_size, S::kPart);
      const int boxes = kTile / rows_per_box;        // of a key tile, and of a part of it:
      const int part_boxes = S::kPart / rows_per_box;
      constexpr int kParts = kTile / S::kPart;
      constexpr int kRing = kE4m3 ? S::kRawUnits : S::kUnits;
      uint64_t* full = kE4m3 ? sm.raw_full : sm.full;
      uint64_t* empty = kE4m3 ? sm.raw_empty : sm.empty;
      int step = 0, item = 0, put = 0;               // put: parts requested
      int queries[2] = {0, 0};                       // row tiles requested
      while (w.left > 0 && ok) {
        // token rows of a row tile are rows tok G + g of its panels
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t == 1 && (!kPair || w.token0 + per_tile >= w.r.n)) break;
          if (queries[t] > 0) ok = __all_sync(0xffffffffu, ok && mbar_wait(&sm.q_empty[t], (queries[t] - 1) & 1));
          if (!ok) break;
          ++queries[t];
          if (lane == 0) {
            mbar_expect_tx(&sm.q_full[t], S::kPanels * per_tile * p.G * 128);
#pragma unroll
            for (int pn = 0; pn < S::kPanels; ++pn)
              tma_load_3d(sm.q[t % S::kQTiles] + pn * kM * 128, &q_map, &sm.q_full[t], pn * 64, w.h * p.G,
                          w.r.t0 + w.token0 + t * per_tile);
          }
          __syncwarp();
        }
        const int count = w.count();
        const int pos0 = w.r.L - w.r.n;
        const int begin = seen_lo(p, max(0, pos0));                       // of the request
        const int lo = seen_lo(p, max(0, pos0 + w.token0));               // of the item
        const int last_pos = pos0 + min(w.r.n, w.token0 + pair) - 1;
        const int hi = min(seen_hi(p, last_pos, w.r.L), w.r.L);
        const int32_t* table = p.c.page_table + (size_t)w.b * p.c.max_pages;
        const int box_first = (w.span.first + w.tile) * boxes;
        int page = 0;
        for (int i = 0; i < count && ok; ++i, ++step) {
          const int in = (i * boxes) & 31;
          if (in == 0) {  // lanes hold the pages of the next 32 boxes
            const int pos = (box_first + i * boxes + lane) * rows_per_box;
            page = -1;
            if (pos < hi && pos + rows_per_box > lo) {
              page = fresh(table + pos / p.c.page_size);
              if (page < 0 || page >= p.c.num_pages) {
                if (pos < (w.span.first + w.tile + count) * kTile) raise_status(p.dev_status, KDA_DEV_BAD_PAGE);
                page = -1;
              }
            }
          }
          const int start = (w.span.first + w.tile + i) * kTile;
          StepNote& note = sm.note[step % kSteps];
#pragma unroll 1
          for (int q = 0; q < 2 * kParts; ++q, ++put) {
            const int kv = q / kParts, part = q % kParts, s = put % kRing;
            if (put >= kRing) ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], (put / kRing - 1) & 1));
            if (!ok) break;
            if (q == 0 && lane == 0) {
              note.flags = (i == 0 ? kFirst : 0) | (i + 1 == count ? kLast : 0) |
                           (w.token0 + per_tile < w.r.n ? kSecond : 0) |
                           (sees_whole<kTree>(p, w.r.L, w.r.n, pos0 + w.token0, last_pos, start) ? kWhole : 0);
              note.start = start;
              note.begin = begin;
              note.end = w.r.L;
              note.item = item;
              note.index = i;
            }
            const int box = part * part_boxes + min(lane, part_boxes - 1);
            const int box_page = __shfl_sync(0xffffffffu, page, in + box);
            const int off = (start + box * rows_per_box) % p.c.page_size;
            const int row = box_page >= 0 ? (box_page * p.c.HKV + w.h) * p.c.page_size + off
                                          : p.c.num_pages * p.c.HKV * p.c.page_size;  // past the end: zeros
            uint32_t bytes = kE4m3 ? S::kRawBytes : S::kUnitBytes;
            if (kE4m3) {
              const unsigned real = __ballot_sync(0xffffffffu, lane < part_boxes && box_page >= 0);
              bytes += __popc(real) * rows_per_box * 4;
              if (lane < part_boxes && box_page < 0) {  // scales of positions without a page are zeros
                for (int j = 0; j < rows_per_box; ++j) sm.raw_scale[s][lane * rows_per_box + j] = 0.f;
                fence_proxy_async_smem();
              }
            }
            __syncwarp();
            if (lane == 0) mbar_expect_tx(&full[s], bytes);
            __syncwarp();
            if (lane < part_boxes) {
              const CUtensorMap* map = kv ? &v_map : &k_map;
              if (kE4m3) {
                tma_load_2d(sm.raw[s] + lane * rows_per_box * D, map, &full[s], 0, row);
                if (box_page >= 0)
                  bulk_load(&sm.raw_scale[s][lane * rows_per_box], (kv ? p.c.v_scale : p.c.k_scale) + row,
                            rows_per_box * 4, &full[s]);
              } else {
#pragma unroll
                for (int pn = 0; pn < S::kPanels; ++pn)
                  tma_load_2d(sm.unit[s] + pn * kTile * 128 + lane * rows_per_box * 128, map, &full[s], pn * 64, row);
              }
            }
          }
        }
        ++item;
        w.next(p, pair, lane);
      }
      if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
      // Every copy lands before the CTA's memory is released, also when a wait gave up.
      for (int u = max(0, put - kRing); u < put; ++u) mbar_wait(&full[u % kRing], (u / kRing) & 1);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (queries[t] > 0) mbar_wait(&sm.q_full[t], (queries[t] - 1) & 1);
    } else if (warp < kMmaWarp + 2) {
      // ---- the products of a slot: the warp waits together, one elected lane issues.
      // Both warps pass every step, and say of every K, V and Q when they are done with it.
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
      const int all = __shfl_sync(0xffffffffu, steps, 0);
      const int slot = __shfl_sync(0xffffffffu, warp, 0) - kMmaWarp;
      const uint32_t s_col = base + slot * kTile, o_col = base + S::kColO + slot * D;
      const uint32_t p_col = base + (slot ? S::col_p(1) : S::col_p(0));
      const uint32_t q0 = smem_u32(sm.q[0]), unit0 = smem_u32(sm.unit[0]);
      auto wait = [&](uint64_t* bar, int parity) { return wait_together(smem_u32(bar), parity); };
      // The slot's next S, found before the turn in which it is issued (if its operands are
      // there by then: PV does not wait for them): its ring place, the step's flags and the
      // addresses of its operands.
      int sg = 0, su = 0, su_phase = 0, s_task = 0, q_items[2] = {0, 0};
      bool q_due = false;   // the item's queries have not been waited for
      bool found = false;
      int f_unit = 0, f_flags = 0;
      uint32_t f_q = 0, f_k = 0;
      auto there = [&](uint64_t* bar, int parity, bool stay) {
        // (a try_wait may put the warp to sleep, and PV would wait)
        if (__all_sync(0xffffffffu, mbar_try(smem_u32(bar), parity))) return true;
        if (stay) ok = wait_on(smem_u32(bar), parity);
        return stay && ok;
      };
      bool counted = false;  // the step's flags have been taken in
      auto find_scores = [&](bool stay) {
        while (sg < all && !found) {
          if (!there(&sm.full[su], su_phase, stay)) return;
          f_flags = __shfl_sync(0xffffffffu, sm.note[sg % kSteps].flags, 0);
          const bool two = kPair && (f_flags & kSecond) != 0;
          if ((f_flags & kFirst) && !counted) {
            q_due = true;
            ++q_items[0];
            if (two) ++q_items[1];
          }
          counted = true;
          if (two || (s_task & 1) == slot) {
            const int tile = two ? slot ^ (s_task & 1) : 0;
            if (q_due && !there(&sm.q_full[tile], ((tile ? q_items[1] : q_items[0]) - 1) & 1, stay)) return;
            q_due = false;
            found = true;
            f_unit = su;
            f_q = q0 + tile * (kM * D * 2);
            f_k = unit0 + su * S::kUnitBytes;
          } else if (elect_one()) {
            mbar_arrive(&sm.empty[su]);
            if (f_flags & kLast) mma_commit(&sm.q_empty[0]);
          }
          __syncwarp();
          counted = false;
          s_task += two ? 2 : 1;
          ++sg;
          su += 2;
          if (su >= S::kUnits) {
            su -= S::kUnits;
            su_phase ^= 1;
          }
        }
      };
      // by the elected lane, after a fence
      auto issue_found = [&](uint64_t* turn) {
        issue_scores<D>(s_col, f_q, f_k, turn);
        mma_commit(&sm.s_full[slot]);
        mma_commit(&sm.empty[f_unit]);
        if (f_flags & kLast) {
          mma_commit(&sm.q_empty[0]);
          if (kPair && (f_flags & kSecond)) mma_commit(&sm.q_empty[1]);
        }
      };
      auto find_and_issue = [&]() {
        find_scores(true);
        if (!ok || !found) return;
        tc_fence_after();
        if (elect_one()) issue_found(nullptr);
        __syncwarp();
        found = false;
      };
      find_and_issue();
      int task = 0, mine = 0, v = 1, v_phase = 0;
      for (int g = 0; g < all && ok; ++g) {
        // (the fixing warp waits for V)
        ok = kE4m3 ? wait(&sm.full[v], v_phase) : wait(&sm.fixed[g % kSteps], (g / kSteps) & 1);
        if (!ok) break;
        const bool two = kPair && (__shfl_sync(0xffffffffu, sm.note[g % kSteps].flags, 0) & kSecond) != 0;
        // the slot's first task of the item starts O
        const bool add = __shfl_sync(0xffffffffu, sm.note[g % kSteps].index, 0) > (two ? 0 : 1);
        if (two || (task & 1) == slot) {
          const uint32_t v_addr = unit0 + v * S::kUnitBytes;
          // task 0 has the first turn; every other one follows the task before it
          find_scores(false);
          ok = wait(&sm.p_half[slot], mine & 1);
          const int first_turn = slot == 0 ? 1 : 0;
          if (ok && mine >= first_turn) ok = wait(&sm.turn[slot], (mine - first_turn) & 1);
          if (!ok) break;
          tc_fence_after();
          // (e4m3 hands the second half over first)
          if (elect_one()) issue_output<D, kE4m3 ? 1 : 0>(o_col, p_col, v_addr, add);
          __syncwarp();
          ok = wait(&sm.p_full[slot], mine & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_output<D, kE4m3 ? 0 : 1>(o_col, p_col, v_addr, true);
            mma_commit(&sm.o_done[slot]);
            mma_commit(&sm.empty[v]);
            if (found) issue_found(&sm.turn[slot ^ 1]);
            else mbar_arrive(&sm.turn[slot ^ 1]);
          }
          __syncwarp();
          ++mine;
          if (found) found = false;
          else find_and_issue();
        } else if (elect_one()) {
          mbar_arrive(&sm.empty[v]);
        }
        __syncwarp();
        task += two ? 2 : 1;
        v += 2;
        if (v >= S::kUnits) {
          v -= S::kUnits;
          v_phase ^= 1;
        }
      }
      if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
      if (elect_one()) mma_commit(&sm.done);  // arrives when every product issued has completed
      __syncwarp();
      mbar_wait(&sm.done, 0);
      __syncwarp();
    } else if (!kE4m3) {
      // ---- entries of V that are not part of the request or not finite, in key tiles
      // that some row sees in part
      for (int g = 0; g < steps && ok; ++g) {
        // K too: a wait for a place's next phase says nothing while the one before it is open,
        // and with an odd number of places V follows K there
        const int u = 2 * g + 1, s = u % S::kUnits;
        ok = mbar_wait(&sm.full[(u - 1) % S::kUnits], ((u - 1) / S::kUnits) & 1) &&
             mbar_wait(&sm.full[s], (u / S::kUnits) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const StepNote& n = sm.note[g % kSteps];
        if ((n.flags & kFirst) && lane == 0) sm.bad[n.item % kSteps] = 0;
        __syncwarp();
        if (!(n.flags & kWhole)) {
          constexpr int kChunks = S::kPanels * kTile * 8;  // of 16 bytes, eight to a panel's row
          const int from = n.begin - n.start, to = n.end - n.start;  // the request's rows
          auto chunk = [&](int i) {
            return reinterpret_cast<uint4*>(sm.unit[s] + (i / (8 * kTile)) * kTile * 128 +
                                            swizzled<128>((i >> 3) & (kTile - 1), i & 7));
          };
          if (from > 0 || to < kTile) {
#pragma unroll 1
            for (int i = lane; i < kChunks; i += 32) {
              const int row = (i >> 3) & (kTile - 1);
              if (row < from || row >= to) *chunk(i) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
          }
          // 0 x is 0 for all that is finite, so that a sum tells: loads and little else (with a
          // look at every entry's exponent the item's last step waited 9000 cycles for this)
          const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
          __nv_bfloat162 sum[4] = {zero, zero, zero, zero};
#pragma unroll 1
          for (int first = lane; first < kChunks; first += 8 * 32) {
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
          const bool any = __any_sync(0xffffffffu, __hisnan(all.x) || __hisnan(all.y));
          if (any) {
#pragma unroll 1
            for (int i = lane; i < kChunks; i += 32) {
              uint4 x = *chunk(i);
              const uint4 out = make_uint4(not_finite(x.x), not_finite(x.y), not_finite(x.z), not_finite(x.w));
              if (out.x | out.y | out.z | out.w)
                *chunk(i) = make_uint4(x.x & ~out.x, x.y & ~out.y, x.z & ~out.z, x.w & ~out.w);
            }
          }
          if (any) sm.bad[n.item % kSteps] = 1;
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.fixed[g % kSteps]);
      }
      if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
    }
  } else {
    // ---- the softmax: one row per thread
    more_registers<S::kSoftmaxRegs>();
    const int t = warp >> 2, r = tid & (kM - 1);
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = lanes + t * kTile, o_col = lanes + S::kColO + t * D, p_col = lanes + S::col_p(t);
    const float c = p.scale * kLog2E;
    const int tok_in = r / p.G, g_in = r - tok_in * p.G;
    const float2 c2 = make_float2(c, c);
    Walk w;
    if (steps > 0) w.start(p, pair, sm.edge[0], steps, lane);
    else w.left = 0;
    int g0 = 0, task0 = 0;   // steps and tasks of the CTA before the item
    int mine = 0, joins = 0; // tasks of this slot so far, items joined so far
    long long item_unit = sm.edge[0].item_unit;
    for (int item = 0; w.left > 0 && ok; ++item, item_unit += S::kItemCost + w.span.tiles, w.next(p, pair, lane)) {
      const int count = w.count(), L = w.r.L, n = w.r.n;
      const bool two = kPair && w.token0 + per_tile < n;
      const int slot0 = task0 & 1;              // the slot of the item's first task
      // two row tiles: this slot has one of them, all steps; one: every other step
      const int tile = two ? t ^ slot0 : 0;
      const int step1 = two ? 0 : t ^ slot0, step_by = two ? 1 : 2;
      const int token0 = w.token0 + tile * per_tile;
      const int token = token0 + tok_in, pos = L - n + token;
      const int row_lo = seen_lo(p, pos), row_hi = min(seen_hi(p, pos, L), L);
      const int tile_first = L - n + token0, tile_last = L - n + min(n, token0 + per_tile) - 1;
      const int start0 = (w.span.first + w.tile) * kTile;
      // the masks of a tree's tokens (rows beyond it have a token's, and are not written)
      auto words_of = [&](int of) { return p.tree + (size_t)(w.r.t0 + min(of, n - 1)) * p.tree_words; };
      [[maybe_unused]] const int32_t* words = kTree ? words_of(token) : nullptr;
      // A row of no token holds what was there before: its maximum never grows, so that it has no say in when the
      // warp rescales.
      auto least = [&](int in) { return in / p.G < per_tile && token0 + in / p.G < n ? -INFINITY : INFINITY; };
      float m = least(r);
      float2 l2 = make_float2(0.f, 0.f);
      bool begun = false;
      [[maybe_unused]] bool rounds = false;  // a maximum of the warp's is past kRounds
      // e4m3: the four rows of the fragment layout, 8 k + lane / 4 of the warp's 32
      [[maybe_unused]] float m4[4], l4[4];
      [[maybe_unused]] int lo4[4], hi4[4];
      if constexpr (kE4m3) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = L - n + token0 + (32 * (warp & 3) + 8 * k + (lane >> 2)) / p.G;
          lo4[k] = seen_lo(p, at);
          hi4[k] = min(seen_hi(p, at, L), L);
          m4[k] = least(32 * (warp & 3) + 8 * k + (lane >> 2));
          l4[k] = 0.f;
        }
      }
      for (int i = step1; i < count; i += step_by, ++mine) {
        const int g = g0 + i;
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[t], mine & 1));
        if (!ok) break;
        tc_fence_after();
        const int start = start0 + i * kTile;
        // whole key tiles of a bf16 cache take x = c S in one product with the subtraction
        const bool whole = sees_whole<kTree>(p, L, n, tile_first, tile_last, start);
        const bool plain = !kE4m3 && whole && c >= 0.f;
        // Scores of 32 columns from col on in units of log 2; what is not seen: -infinity.
        auto scored = [&](float(&x)[32], int col) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float2 a = __fmul2_rn(make_float2(x[e], x[e + 1]), c2);
            const float2 b = __fmul2_rn(make_float2(x[e + 2], x[e + 3]), c2);
            x[e] = a.x;
            x[e + 1] = a.y;
            x[e + 2] = b.x;
            x[e + 3] = b.y;
          }
          if (!whole) {
            uint32_t see = columns(row_lo - start - col, row_hi - start - col);
            if (kTree) see &= tree_bits(words, p.tree_words, n, start + col - (L - n));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1)) x[e] = -INFINITY;
          }
        };
        auto highest = [](const float(&x)[32]) {
          float y = fmaxf(x[0], x[1]), z = fmaxf(x[2], x[3]);
#pragma unroll
          for (int e = 4; e < 32; e += 4) {
            y = max3(y, x[e], x[e + 1]);
            z = max3(z, x[e + 2], x[e + 3]);
          }
          return fmaxf(y, z);
        };
        // A larger maximum moves the sum and O; S came after the product before it, so O is
        // at rest.
        auto move = [&](float top) {
          const float now = fmaxf(m, top);
          if (__any_sync(0xffffffffu, now > m + kGrow)) {
            const float keep = exp2_approx(m - (now == -INFINITY ? 0.f : now));
            l2.x *= keep;
            l2.y *= keep;
            if (begun) {
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
            rounds = __any_sync(0xffffffffu, fabsf(m) > kRounds && fabsf(m) < INFINITY);
          }
          begun = true;
        };
        float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
        // The weights of 32 columns as bf16 pairs, to TMEM.
        auto weigh = [&](const float(&x)[32], int col, auto is_plain) {
          const float ref = m == -INFINITY ? 0.f : m;
          const float2 nref = make_float2(-ref, -ref);
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float2 xa = make_float2(x[e], x[e + 1]), xb = make_float2(x[e + 2], x[e + 3]);
            const float2 ya = decltype(is_plain)::value ? __ffma2_rn(xa, c2, nref) : __fadd2_rn(xa, nref);
            const float2 yb = decltype(is_plain)::value ? __ffma2_rn(xb, c2, nref) : __fadd2_rn(xb, nref);
            const float2 va = make_float2(exp2_approx(ya.x), exp2_approx(ya.y));
            const float2 vb = make_float2(exp2_approx(yb.x), exp2_approx(yb.y));
            sum0 = __fadd2_rn(sum0, va);
            sum1 = __fadd2_rn(sum1, vb);
            pw[e / 2] = pack_bf16(va.x, va.y);
            pw[e / 2 + 1] = pack_bf16(vb.x, vb.y);
          }
          tmem_st_16cols(p_col + col / 2, pw);
        };
        auto hand_over = [&](uint64_t* bar) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        };
        if constexpr (!kE4m3) {
          // all of S in registers
          float x[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld_32cols(s_col + 32 * q, x[q]);
          tmem_ld_wait();
          if (!plain)
#pragma unroll
            for (int q = 0; q < 4; ++q) scored(x[q], 32 * q);
          const float top = fmaxf(max3(highest(x[0]), highest(x[1]), highest(x[2])), highest(x[3]));
          move(plain ? top * c : top);
          // x = c S is exact in the one product and the maximum rounded, by hundreds where scores
          // are billions: there both are rounded, so that the largest weight is 1
          const bool fused = plain && !rounds;
          if (__builtin_expect(plain && rounds, 0)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) scored(x[q], 32 * q);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (fused) weigh(x[q], 32 * q, std::true_type{});
            else weigh(x[q], 32 * q, std::false_type{});
            if (q == 1) hand_over(&sm.p_half[t]);
          }
          hand_over(&sm.p_full[t]);
        } else {
          // A key's and a value's scale belong to a column, so the fragment layout is taken, in
          // which a thread has a quarter of the columns of four rows: a quarter of the loads
          // of scales (with a row to a thread they took 5000 cycles a task).  Half of S in
          // registers; the first half is read again after the second.
          const float* k_scale = sm.scale[g % S::kScaleSteps][0] + 2 * (lane & 3);
          const float* v_scale = sm.scale[g % S::kScaleSteps][1] + 2 * (lane & 3);
          float x[2][32];
          auto load = [&](int col) {
            tmem_ld_fragments_64cols(s_col + col, x[0]);
            tmem_ld_fragments_64cols(s_col + col + (16u << 16), x[1]);
            tmem_ld_wait();
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const float2 f = *reinterpret_cast<const float2*>(k_scale + col + 8 * b);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float* y = &x[k >> 1][4 * b + 2 * (k & 1)];
                const float2 z = __fmul2_rn(make_float2(y[0], y[1]), f);
                y[0] = z.x;
                y[1] = z.y;
              }
            }
            if (!whole) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int at = start + col + 2 * (lane & 3);
                const int from = lo4[k] - at, to = hi4[k] - at;  // seen: from <= 8 b + e < to
                [[maybe_unused]] uint32_t tree[2];
                if constexpr (kTree) {
                  const int32_t* of = words_of(token0 + (32 * (warp & 3) + 8 * k + (lane >> 2)) / p.G);
                  tree[0] = tree_bits(of, p.tree_words, n, at - (L - n));
                  tree[1] = tree_bits(of, p.tree_words, n, at + 32 - (L - n));
                }
#pragma unroll
                for (int b = 0; b < 8; ++b)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    bool hidden = 8 * b + e < from || 8 * b + e >= to;
                    if constexpr (kTree) hidden |= !((tree[b >> 2] >> (8 * (b & 3) + e)) & 1);
                    if (hidden) x[k >> 1][4 * b + 2 * (k & 1) + e] = -INFINITY;
                  }
              }
            }
          };
          float now[4] = {m4[0], m4[1], m4[2], m4[3]};
          auto raise = [&]() {
#pragma unroll
            for (int b = 0; b < 8; ++b)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                now[k] = max3(now[k], x[k >> 1][4 * b + 2 * (k & 1)], x[k >> 1][4 * b + 2 * (k & 1) + 1]);
          };
          load(0);
          raise();
          load(64);
          raise();
          bool grown = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            now[k] = fmaxf(now[k], __shfl_xor_sync(0xffffffffu, now[k], 1));
            now[k] = fmaxf(now[k], __shfl_xor_sync(0xffffffffu, now[k], 2));
            grown |= now[k] > m4[k] + kGrow;
          }
          if (__any_sync(0xffffffffu, grown)) {
            float keep[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              keep[k] = exp2_approx(m4[k] - (now[k] == -INFINITY ? 0.f : now[k]));
              l4[k] *= keep[k];
              m4[k] = now[k];
            }
            if (begun) {
#pragma unroll 1
              for (int cc = 0; cc < 2 * D; cc += 32) {  // 16 lanes, then the others
                const uint32_t at = o_col + cc % D + (cc >= D ? 16u << 16 : 0u);
                float o[16];
                tmem_ld_fragments_32cols(at, o);
                tmem_ld_wait();
                uint32_t ob[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  ob[e] = __float_as_uint(o[e] * ((e >> 1) & 1 ? (cc >= D ? keep[3] : keep[1])
                                                               : (cc >= D ? keep[2] : keep[0])));
                tmem_st_fragments_32cols(at, ob);
              }
            }
          }
          begun = true;
          float nref[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) nref[k] = m4[k] == -INFINITY ? 0.f : -m4[k];
          auto weigh4 = [&](int col, auto is_whole) {
            uint32_t pw[2][16];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const float2 f = *reinterpret_cast<const float2*>(v_scale + col + 8 * b);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float* y = &x[k >> 1][4 * b + 2 * (k & 1)];
                const float2 z = __fadd2_rn(make_float2(y[0], y[1]), make_float2(nref[k], nref[k]));
                float2 v = make_float2(exp2_approx(z.x), exp2_approx(z.y));
                l4[k] += v.x + v.y;
                v = __fmul2_rn(v, f);
                if constexpr (!decltype(is_whole)::value) {
                  // a weight of 0 stays 0 whatever the scale of a place that is not seen
                  if (y[0] == -INFINITY) v.x = 0.f;
                  if (y[1] == -INFINITY) v.y = 0.f;
                }
                pw[k >> 1][2 * b + (k & 1)] = pack_bf16(v.x, v.y);
              }
            }
            tmem_st_packed_fragments_32cols(p_col + col / 2, pw[0]);
            tmem_st_packed_fragments_32cols(p_col + col / 2 + (16u << 16), pw[1]);
          };
          const int u = 2 * g + 1;  // V's scales are written with V
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[u % S::kUnits], (u / S::kUnits) & 1));
          if (!ok) break;
          if (whole) weigh4(64, std::true_type{});
          else weigh4(64, std::false_type{});
          hand_over(&sm.p_half[t]);
          load(0);
          if (whole) weigh4(0, std::true_type{});
          else weigh4(0, std::false_type{});
          hand_over(&sm.p_full[t]);
        }
        if constexpr (!kE4m3) l2 = __fadd2_rn(l2, __fadd2_rn(sum0, sum1));
      }
      const int first_join = joins;
      if (!two && count > 1) ++joins;
      g0 += count;
      task0 += two ? 2 * count : count;
      if (!ok) break;
      if (!begun) continue;  // the only step was the other slot's
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_done[t], (mine - 1) & 1));
      if (!ok) break;
      // ---- the end of this CTA's part of the item
      tc_fence_after();
      float l = l2.x + l2.y;
      if constexpr (kE4m3) {  // to a row per thread (the warp's own 32)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          l4[k] += __shfl_xor_sync(0xffffffffu, l4[k], 1);
          l4[k] += __shfl_xor_sync(0xffffffffu, l4[k], 2);
          if ((lane & 3) == 0) sm.rows[t][32 * (warp & 3) + 8 * k + (lane >> 2)] = make_float2(m4[k], l4[k]);
        }
        __syncwarp();
        m = sm.rows[t][r].x;
        l = sm.rows[t][r].y;
        __syncwarp();
      }
      float keep = 1.f, keep2 = 0.f;
      const bool join = !two && count > 1;
      if (join) {
        if (t != slot0) {
          // the second slot hands its sums over, and keeps its O until it has been read
          sm.other[r] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.join_ready);
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.join_done, first_join & 1));
          if (!ok) break;
          tc_fence_after();
          continue;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.join_ready, first_join & 1));
        if (!ok) break;
        tc_fence_after();
        const float2 ml = sm.other[r];
        const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
        keep = exp2_approx(m - ref);
        keep2 = exp2_approx(ml.x - ref);
        l = l * keep + ml.y * keep2;
        m = top;
      }
      const uint32_t o_other = lanes + S::kColO + (t ^ 1) * D;
      const bool begins = w.tile == 0, ends = w.tile + count == w.span.tiles;
      const bool done = begins && ends;
      const bool live = tok_in < per_tile && token < n;
      const size_t out_row = (size_t)(w.r.t0 + token) * p.H + w.h * p.G + g_in;
      int to_rows[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) to_rows[e] = __shfl_sync(0xffffffffu, live ? (int)out_row : -1, (lane & ~3) + e);
      const size_t piece = ((size_t)cta * 2 + (begins ? 1 : 0)) * kChunkRows + tile * per_tile * p.G + r;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool bad = !kE4m3 && sm.bad[item % kSteps] != 0;
      if (live) {
        if (!done) pieces.ml[piece] = make_float2(m, l);
        else if (p.lse) p.lse[out_row] = (m + log2f(l)) * kLn2;
      }
      if (r == 0 && t == slot0 && begins && !ends)
        pieces.notes[cta] = PieceNote{(w.r.t0 + w.token0) * p.H + w.h * p.G, min(pair, n - w.token0),
                                      share_of(units, used, item_unit + S::kItemCost + w.span.tiles - 1) - cta + 1, 0};
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 32) {
        float o[32];
        tmem_ld_32cols(o_col + cc, o);
        tmem_ld_wait();
        if (join) {
          float o2[32];
          tmem_ld_32cols(o_other + cc, o2);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(o[e], keep, o2[e] * keep2);
        }
        if (live && bad) {
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = o[e];
          add_bad_values<D, kTree>(p, w.b, w.h, L, n, pos, L - n + w.token0, L - n + min(n, w.token0 + pair) - 1,
                            start0, count, words, p.q + (w.r.t0 + token) * p.q_stride + (size_t)(w.h * p.G + g_in) * D,
                            m == -INFINITY ? 0.f : m, cc, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = y[e];
        }
        if (done) {
          uint4 y[4];
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            y[e / 8] = make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                                  pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
          // four lanes write 64 bytes of one row together
          transpose4(y, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (to_rows[e] >= 0) *reinterpret_cast<uint4*>(p.out + (size_t)to_rows[e] * D + cc + 8 * (lane & 3)) = y[e];
          }
        } else if (live) {
          float4* to = reinterpret_cast<float4*>(pieces.o + piece * D + cc);
#pragma unroll
          for (int e = 0; e < 32; e += 4) to[e / 4] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        __syncwarp();  // the next load is the whole warp's
      }
      if (join) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.join_done);
      }
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool kE4m3, bool kPair, bool kTree>
cudaError_t launch_chunk(const AttentionArgs& a, cudaStream_t stream) {
  using Sm = Smem<D, kE4m3, kPair>;
  using S = Shape<D, kE4m3, kPair>;
  static_assert(sizeof(Sm) + 1024 <= 227 * 1024, "a chunk CTA fits an SM");
  CUtensorMap q_map, maps[2];
  const int per_tile = kM / a.G;
  if (!make_map_3d_bf16(&q_map, a.q, D, a.H, a.T, D * 2, (uint64_t)a.q_stride * 2, 64, a.G, per_tile))
    return cudaErrorInvalidValue;
  const uint64_t rows = (uint64_t)a.c.num_pages * a.c.HKV * a.c.page_size;
  for (int i = 0; i < 2; ++i)
    if (!make_map_2d(&maps[i], kE4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     kE4m3 ? 1 : 2, i ? a.c.v : a.c.k, D, rows, kE4m3 ? D : 64,
                     a.c.page_size < S::kPart ? a.c.page_size : S::kPart,
                     kE4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  const size_t smem = sizeof(Sm) + 1024;
  static SmemSet set;
  cudaError_t e = allow_smem(chunk_kernel<D, kE4m3, kPair, kTree>, smem, set);
  if (e != cudaSuccess) return e;
  const Pieces pieces = pieces_at(a.workspace, kChunkCtas, kChunkRows);
  e = launch(chunk_kernel<D, kE4m3, kPair, kTree>, dim3(kChunkCtas), dim3(S::kThreads), smem, stream, true, q_map,
             maps[0], maps[1], a, pieces);
  if (e != cudaSuccess) return e;
  return launch_join_pieces(a, pieces, kChunkRows, kChunkCtas, stream);
}

template <bool kTree, int D, bool kE4m3>
cudaError_t by_pair(const AttentionArgs& a, cudaStream_t stream) {
  return a.max_tokens > kM / a.G ? launch_chunk<D, kE4m3, true, kTree>(a, stream)
                                 : launch_chunk<D, kE4m3, false, kTree>(a, stream);
}

}  // namespace
}  // namespace kda
