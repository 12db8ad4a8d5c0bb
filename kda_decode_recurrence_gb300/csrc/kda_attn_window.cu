// kda_attn_window.cu -- attention of single tokens and drafted windows: the requests
// with few rows (new tokens x query heads per key head: window_limit).
//
// Such a request reads every cached row for 4 G n_b operations a byte at most, so HBM
// bounds it and the kernel is built to keep copies in flight: two or three CTAs per
// SM, each with a ring of key tiles (64 positions of K and V) filled by one
// warp through TMA, one box per page and 128-byte panel.  Key tiles of all
// requests are divided evenly over the CTAs (kda_attn.cuh), whatever their lengths.
//
// Per key tile the four computing warps split first the positions, then the
// head dimension:
//   S[rows, 16 w .. 16 w + 15] = Q K^T        warp w's 16 positions
//   the rows' maxima are exchanged through shared memory, P = 2^(S - m) goes
//   there in V's type (the instruction takes one for both), bf16 here
//   O[rows, D/4 w ..] = O 2^(m_old - m) + P V  warp w's quarter of D
// so that each entry of K and V is read from shared memory (and, for e4m3,
// widened) once, and no warp's output has to be joined with another's.
// e4m3 codes are widened to f16 (one conversion for two; bf16 takes five operations on
// the pipe that is busiest), so Q and P are f16 there too.  Q is scaled by a power of two
// per item (its largest entry becomes 2^8 .. 2^9) and exact: an item with entries too small
// for f16 beside that one (26 octaves below it) keeps Q in bf16, and its codes of K are widened
// to bf16.  P is scaled by a power of two per CTA's part of an item:
//   w_j = 2^(x_j - m),  P_j = F w_j vs_j   (vs_j: the value's scale)
// F takes the first key tile's largest vs to 2^7 .. 2^8; as long as every F vs_j that is not
// 0 lies in 2^0 .. 2^15, P is within f16 and its error within 2^-11 of it or 2^-25 of the
// largest weight (bf16: 2^-8).  Scales that do not fit (a row of zeros beside tiny values
// has the scale 1) end that for the rest of the part: P is then w_j vs_j in bf16, whose range
// is fp32's, and the codes of V are widened to bf16.  (log2 vs_j in the reference, in place of
// F, lets scales of rows without weight take bits from the others, and next to scores of 2^24
// it rounds by octaves.)
// mma.sync (m16n8k16) is the instruction for it: 16 rows are its native
// size, where tcgen05 would spend 128 lanes on them.
//
// 128 single tokens over 5.05 GB of bf16 cache: 713 us, 7.07 TB/s (a copy: 6.70).
// 64 over 628 MB of e4m3: 146 us, 4.30 TB/s (142 without the look at V's scales; two CTAs an SM
// and bf16 operands throughout: 178; P in bf16 177, Q 206, both 237).  Its schedulers issue in 49% of the cycles, with three
// computing warps each, and DRAM is at 55%: what bounds it are the tile's dependent steps (per
// instruction 2.0 cycles of fixed latencies, 1.7 of loads, 0.6 at barriers, of 7.4).
// With more rows a warp reads as many operands of Q and P as of K and V: 32 rows are for e4m3
// only (32 such requests, cold L2: 114 us against the chunk kernel's 140).  Eight warps that
// split D by eight: 165 us and 755 us on these two; streams of 32 positions per warp that
// exchange nothing until an item's end, one CTA an SM: 265 us and 1320 us.
#include <cuda.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kda_attn.cuh"
#include "kda_launch.h"
#include "kda_tcgen05.cuh"
#include "kda_tmap.h"

namespace kda {
namespace {

constexpr int kTile = 64;             // positions per key tile
constexpr int kComputeWarps = 4;
constexpr int kThreads = 32 * (kComputeWarps + 2);  // + one warp for K and V, one for Q

struct StageNote {
  int t0, n, L, h;   // the item
  int start;         // first position of the key tile
  int flags;         // kFirst, kLast of this CTA's part of the item; kBegins, kEnds the item
  int pieces;        // CTAs that share the item (flags has kBegins and not kEnds)
  int pad;
};
constexpr int kFirst = 1, kLast = 2, kBegins = 4, kEnds = 8;

template <int D, int kRows, bool kE4m3>
struct Shape {
  static constexpr int kElem = kE4m3 ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;              // 64, 128 or 256
  static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kPanels = kRowBytes / kPanelBytes;
  static constexpr int kTileBytes = kTile * kRowBytes;     // K or V
  // CTAs per SM: e4m3 has twice the tiles for its bytes, and what a warp does per tile is a
  // chain of dependent steps, so a third CTA fills issue slots where the registers allow it
  static constexpr int kCtas = kE4m3 && kRows == 16 ? 3 : 2;
  // the ring: as deep as lets them share the SM
  static constexpr int kOther = 2 * kRows * D * 2 + kRows * kTile * 2 + 4096;
  static constexpr int kStageBytes = 2 * kTileBytes + (kE4m3 ? 2 * kTile * 4 : 0);
  static constexpr int kFit = ((227 * 1024) / kCtas - 1024 - kOther) / kStageBytes;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
};

template <int D, int kRows, bool kE4m3>
struct Smem {
  using S = Shape<D, kRows, kE4m3>;
  unsigned char kv[S::kStages][2][S::kTileBytes];  // 1024-aligned, swizzled panels
  unsigned char q[2][kRows * D * 2];               // rows of 128-byte swizzled panels
  unsigned char pw[kRows * kTile * 2];             // P, bf16, 128-byte swizzled rows
  float scales[kE4m3 ? S::kStages : 1][2][kTile];
  float4 top[kRows];                               // the warps' row maxima
  float qinv[2];                                   // e4m3: what undoes Q's scaling
  int4 span[kComputeWarps];                        // e4m3: of the warps' scales of V (see below)
  int qwide[2];                                    // e4m3: Q is bf16, f16 would lose bits
  StageNote note[S::kStages];
  uint64_t full[S::kStages], empty[S::kStages], qfull[2], qempty[2];
  long long part[kThreads / 32];
  int start_b;
  long long start_unit;
};

__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 codes (the low half of x) as f16 values.
__device__ __forceinline__ uint32_t codes_f16(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// F takes a part's first scales to at most 2^kSpan .. 2^(kSpan + 1) and at least 2^0.  Those
// that fit then lie in 1 / F .. 2^(2 kSpan + 1) / F, kRoom steps of their bits.  (One that is
// not finite makes the rows that see it NaN in either type, and must not show in the others.)
constexpr int kSpan = 7;
constexpr uint32_t kRoom = (uint32_t)(2 * kSpan + 1) << 23, kUnset = 0x80000000u;

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Barriers of the computing warps; the second also says whether all of them go on.
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kComputeWarps) : "memory");
}
__device__ __forceinline__ bool compute_sync_and(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, 1, %2, q;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(all) : "r"((uint32_t)ok), "n"(32 * kComputeWarps) : "memory");
  return all != 0;
}
// Units of a request: 0 if it is not this kernel's, else HKV x its key tiles
// (at least one each: rows that see nothing are written too).
__device__ __forceinline__ int first_tile(const AttentionArgs& p, const Request& r) {
  return seen_lo(p, max(0, r.L - r.n)) / kTile;
}
__device__ __forceinline__ int key_tiles(const AttentionArgs& p, const Request& r) {
  return max(1, (r.L + kTile - 1) / kTile - first_tile(p, r));
}
__device__ __forceinline__ long long units_of(const AttentionArgs& p, const Request& r) {
  return r.n > 0 && r.n * p.G <= p.window_rows ? (long long)p.c.HKV * key_tiles(p, r) : 0;
}

// The items of one CTA's share in order, walked by a whole warp: 32 requests
// are looked up at a time.
struct Walk {
  int base;          // the request that lane 0 holds
  Request mine;      // this lane's request
  int b, h;          // the current item
  Request r;
  int tile, tiles;   // next key tile of the item (0 .. tiles - 1)
  long long left;    // units left in this CTA's share

  __device__ __forceinline__ void fetch(const AttentionArgs& p, int from, int lane) {
    base = from;
    mine = Request{0, 0, 0};
    if (from + lane < p.B) mine = load_request(p, from + lane, false);
    if (units_of(p, mine) == 0) mine.n = 0;
  }
  __device__ __forceinline__ void take(const AttentionArgs& p, int lane) {
    // the first request at b or after it with units
    while (true) {
      if (b >= base + 32) fetch(p, b, lane);
      const unsigned some = __ballot_sync(0xffffffffu, mine.n > 0) & (0xffffffffu << (b - base));
      if (some) {
        const int src = __ffs(some) - 1;
        b = base + src;
        r.t0 = __shfl_sync(0xffffffffu, mine.t0, src);
        r.n = __shfl_sync(0xffffffffu, mine.n, src);
        r.L = __shfl_sync(0xffffffffu, mine.L, src);
        tiles = key_tiles(p, r);
        return;
      }
      b = base + 32;
      if (b >= p.B) {  // cannot happen while units are left
        left = 0;
        return;
      }
    }
  }
  // Start at unit `skip` of request b's.
  __device__ __forceinline__ void start(const AttentionArgs& p, int b0, long long skip, long long units, int lane) {
    b = b0;
    left = units;
    fetch(p, b, lane);
    take(p, lane);
    h = (int)(skip / tiles);
    tile = (int)(skip % tiles);
  }
  // Units of the current item that this CTA takes, from `tile` on.
  __device__ __forceinline__ int count() const { return (int)min((long long)(tiles - tile), left); }
  __device__ __forceinline__ void next(const AttentionArgs& p, int lane) {
    left -= count();
    if (left <= 0) return;
    tile = 0;
    if (++h == p.c.HKV) {
      h = 0;
      ++b;
      take(p, lane);
    }
  }
};

template <int D, int kRows, bool kE4m3>
__global__ void __launch_bounds__(kThreads, Shape<D, kRows, kE4m3>::kCtas)
    window_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const AttentionArgs p, const Pieces pieces) {
  using S = Shape<D, kRows, kE4m3>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D, kRows, kE4m3>& sm = *reinterpret_cast<Smem<D, kRows, kE4m3>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;

  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], kComputeWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.qfull[s], 1);
      mbar_init(&sm.qempty[s], kComputeWarps);
    }
    mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share: each thread counts a run of requests
  if (cta == 0 && tid == kThreads - 1) check_offsets(p);
  const int run = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(p.B, tid * run), b_hi = min(p.B, b_lo + run);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += units_of(p, load_request(p, b, cta == 0));
  long long units;
  const long long from = scan_before<kThreads / 32>(mine, sm.part, units);
  const int used = (int)min((long long)ctas, units);
  if (tid == 0) pieces.notes[cta].tokens = 0;
  if (cta >= used) return;
  const long long u0 = share_begin(units, used, cta), u1 = share_begin(units, used, cta + 1);
  if (u0 >= from && u0 < from + mine) {
    long long at = from;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long u = units_of(p, load_request(p, b, false));
      if (u0 < at + u) {
        sm.start_b = b;
        sm.start_unit = u0 - at;
        break;
      }
      at += u;
    }
  }
  __syncthreads();

  if (warp == kComputeWarps) {
    // ---- K and V of every key tile into the ring
    Walk w;
    w.start(p, sm.start_b, sm.start_unit, u1 - u0, lane);
    const int rows_per_box = min(p.c.page_size, kTile);
    const int boxes = kTile / rows_per_box;
    int it = 0;
    long long unit = u0;
    bool ok = true;
    while (w.left > 0 && ok) {
      const int count = w.count();
      const int lo = seen_lo(p, max(0, w.r.L - w.r.n));
      const int t_first = first_tile(p, w.r);
      const int32_t* table = p.c.page_table + (size_t)w.b * p.c.max_pages;
      const int box_first = (t_first + w.tile) * boxes;  // box i of the segment is box_first + i
      int page = 0;
      for (int i = 0; i < count; ++i, ++it) {
        // lanes hold the pages of the next 32 boxes
        const int in = (i * boxes) & 31;
        if (in == 0) {
          const int pos = (box_first + i * boxes + lane) * rows_per_box;
          page = -2;  // no position in use: zeros, no report
          if (pos < w.r.L && pos + rows_per_box > lo) {
            page = fresh(table + pos / p.c.page_size);
            if (page < 0 || page >= p.c.num_pages) {
              if ((long long)pos < (long long)(t_first + w.tile + count) * kTile)
                raise_status(p.dev_status, KDA_DEV_BAD_PAGE);
              page = -1;
            }
          }
        }
        const int s = it % S::kStages;
        if (it >= S::kStages) ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[s], (it / S::kStages - 1) & 1));
        if (!ok) break;
        const int start = (t_first + w.tile + i) * kTile;
        if (lane == 0) {
          StageNote& note = sm.note[s];
          note.t0 = w.r.t0;
          note.n = w.r.n;
          note.L = w.r.L;
          note.h = w.h;
          note.start = start;
          const bool begins = w.tile == 0, ends = w.tile + count == w.tiles;
          note.flags = (i == 0 ? kFirst : 0) | (i + 1 == count ? kLast : 0) | (begins ? kBegins : 0) |
                       (ends ? kEnds : 0);
          note.pieces = begins && !ends ? share_of(units, used, unit + w.tiles - 1) - cta + 1 : 1;
        }
        if (kE4m3) {
          // scales of boxes without a page are zeros; written before the barrier's arrival
          for (int j = lane; j < kTile; j += 32) {
            const int pg = __shfl_sync(0xffffffffu, page, in + j / rows_per_box);
            if (pg < 0) sm.scales[s][0][j] = sm.scales[s][1][j] = 0.f;
          }
          fence_proxy_async_smem();  // a later copy to the same place comes after
        }
        __syncwarp();
        const int mine_page = __shfl_sync(0xffffffffu, page, in + min(lane, boxes - 1));
        const unsigned real = __ballot_sync(0xffffffffu, lane < boxes && mine_page >= 0);
        if (lane == 0)
          mbar_expect_tx(&sm.full[s], 2 * S::kTileBytes + (kE4m3 ? __popc(real) * 2 * rows_per_box * 4 : 0));
        __syncwarp();
        if (lane < boxes) {
          const int off = (start + lane * rows_per_box) % p.c.page_size;
          const int row = mine_page >= 0 ? (mine_page * p.c.HKV + w.h) * p.c.page_size + off
                                         : p.c.num_pages * p.c.HKV * p.c.page_size;  // past the end: zeros
#pragma unroll
          for (int pn = 0; pn < S::kPanels; ++pn) {
            const int at = pn * kTile * S::kPanelBytes + lane * rows_per_box * S::kPanelBytes;
            tma_load_2d(sm.kv[s][0] + at, &k_map, &sm.full[s], pn * (S::kPanelBytes / S::kElem), row);
            tma_load_2d(sm.kv[s][1] + at, &v_map, &sm.full[s], pn * (S::kPanelBytes / S::kElem), row);
          }
          if (kE4m3 && mine_page >= 0) {
            bulk_load(&sm.scales[s][0][lane * rows_per_box], p.c.k_scale + row, rows_per_box * 4, &sm.full[s]);
            bulk_load(&sm.scales[s][1][lane * rows_per_box], p.c.v_scale + row, rows_per_box * 4, &sm.full[s]);
          }
        }
      }
      unit += count;
      w.next(p, lane);
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
    // Every copy lands before the CTA's memory is released, also when a wait gave up.
    for (int i = max(0, it - S::kStages); i < it; ++i)
      mbar_wait(&sm.full[i % S::kStages], (i / S::kStages) & 1);
  } else if (warp == kComputeWarps + 1) {
    // ---- the items' queries into two buffers: row i G + g is token i, head h G + g
    Walk w;
    w.start(p, sm.start_b, sm.start_unit, u1 - u0, lane);
    bool ok = true;
    for (int it = 0; w.left > 0 && ok; ++it) {
      const int s = it & 1;
      if (it >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&sm.qempty[s], (it / 2 - 1) & 1));
      if (!ok) break;
      constexpr int kChunks = D / 8;  // 16-byte chunks of a row
      const int rows = w.r.n * p.G;
      const int padding = max(0, w.r.n - w.r.L) * p.G;  // rows of tokens before position 0: zeros
      auto load = [&](int i) {
        const int row = i / kChunks, c = i % kChunks;
        if (row < padding || row >= rows) return make_uint4(0, 0, 0, 0);
        return *reinterpret_cast<const uint4*>(
            p.q + (w.r.t0 + row / p.G) * p.q_stride + (size_t)(w.h * p.G + row % p.G) * D + c * 8);
      };
      auto store = [&](int i, uint4 x, float factor, bool wide) {
        const int row = i / kChunks, c = i % kChunks;
        unsigned char* to = sm.q[s] + (c / 8) * kRows * 128;
        if constexpr (kE4m3) {
          // Four consecutive entries of K sit in one register of the tensor core's
          // operand, pairs (0 1) (2 3) as k = 2 j .. and 2 j + 8 ..: the same order here.
          // Entries 4 j .. 4 j + 3 of each 16 go to 2 j, 2 j + 1, 2 j + 8, 2 j + 9.
          const int j = (c & 1) * 2;  // this chunk's first group of four
          const int c0 = (c & 7) & ~1;
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = bf16_lo(v[e]) * factor, hi = bf16_hi(v[e]) * factor;
            *reinterpret_cast<uint32_t*>(to + swizzled<128>(row, c0 + (e & 1)) + j * 4 + (e >> 1) * 4) =
                wide ? pack_bf16(lo, hi) : pack_f16(lo, hi);
          }
        } else {
          *reinterpret_cast<uint4*>(to + swizzled<128>(row, c & 7)) = x;
        }
      };
      constexpr int kLoads = kRows * kChunks / 32;
      if constexpr (kE4m3) {
        // the largest finite entry's exponent e: factor 2^(135 - e); the smallest's that is
        // not 0 says whether f16 holds them all (least: its bits less 1, so that 0 is the most)
        uint32_t top = 0, least = 0xffffffffu;
        auto raise = [&](const uint4& x) {
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = v[e] & 0x7fffu, hi = (v[e] >> 16) & 0x7fffu;
            top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            least = min(least, min(lo - 1u, hi - 1u));
          }
        };
        uint4 held[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) held[i] = load(i * 32 + lane);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) raise(held[i]);
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) {
          top = max(top, __shfl_xor_sync(0xffffffffu, top, e));
          least = min(least, __shfl_xor_sync(0xffffffffu, least, e));
        }
        const int field = min(253, 262 - (int)(top >> 7));  // its inverse is a normal number too
        const float factor = __uint_as_float((uint32_t)field << 23);
        // the last bit of the smallest, 2^(e - 134) of its exponent field e (1 for a subnormal),
        // times 2^(field - 127): no smaller than f16's, 2^-24
        const bool wide = least < 0x7f80u && max(1, (int)((least + 1u) >> 7)) + field < 237;
        if (lane == 0) {
          sm.qinv[s] = __uint_as_float((uint32_t)(254 - field) << 23);
          sm.qwide[s] = wide;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) store(i * 32 + lane, held[i], factor, wide);
      } else {
#pragma unroll 8
        for (int i = 0; i < kLoads; ++i) store(i * 32 + lane, load(i * 32 + lane), 1.f, false);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.qfull[s]);
      w.next(p, lane);
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
  } else {
    // ---- the four computing warps
    constexpr int kR = kRows / 16;        // row blocks of 16
    constexpr int kN = D / kComputeWarps / 8;  // blocks of 8 columns of O per warp
    const int quad = lane >> 2, j2 = (lane & 3) * 2;
    float xscale = p.scale * kLog2E;
    [[maybe_unused]] bool q_wide = false;
    float o[kR][kN][4], m[kR][2], l[kR][2];
    // e4m3: F, the bits of 1 / F (kUnset: no scale has been seen, and F is 1), and whether P is
    // bf16 (then F is 1 too)
    [[maybe_unused]] float factor = 1.f;
    [[maybe_unused]] uint32_t unit = kUnset;
    [[maybe_unused]] bool v_wide = false;
    long long left = u1 - u0;
    int item = -1;
    bool ok = true;
    for (int it = 0; left > 0; ++it, --left) {
      const int s = it % S::kStages;
      // A wait that gives up in any of the warps ends all four at the next barrier.
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[s], (it / S::kStages) & 1));
      StageNote note = {};
      if (ok) note = sm.note[s];
      if (note.flags & kFirst) {
        ++item;
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.qfull[item & 1], (item / 2) & 1));
        if (kE4m3) {
          xscale = p.scale * kLog2E * sm.qinv[item & 1];
          q_wide = sm.qwide[item & 1] != 0;
        }
        factor = 1.f;
        unit = kUnset;
        v_wide = false;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          m[r][0] = m[r][1] = -INFINITY;
          l[r][0] = l[r][1] = 0.f;
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[r][n][i] = 0.f;
        }
      }
      const uint32_t k_addr = smem_u32(sm.kv[s][0]), v_addr = smem_u32(sm.kv[s][1]);
      const uint32_t q_addr = smem_u32(sm.q[item & 1]), p_addr = smem_u32(sm.pw);

      const int my_pos = 16 * warp;
      const int pos0 = note.L - note.n;   // position of token 0
      const int lo_all = seen_lo(p, max(0, pos0));
      const bool v_whole = note.start >= lo_all && note.start + kTile <= note.L;  // all seen by some token
      bool narrow = true;
      // the bits of one of the warp's 16 scales of V, each in two lanes
      auto scale_bits = [&]() {
        const int at = my_pos + (lane & 15);
        const uint32_t bits = __float_as_uint(sm.scales[s][1][at]) & 0x7fffffffu;
        return !v_whole && (note.start + at < lo_all || note.start + at >= note.L) ? 0u : bits;
      };
      if constexpr (kE4m3) {
        const uint32_t bits = scale_bits();
        narrow = v_wide | (bits == 0) | (bits - unit < kRoom);
      }

      // S: this warp's 16 positions x all rows
      float x[kR][2][4];
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[r][n][i] = 0.f;
      auto dot16 = [&](int kb, uint32_t b00, uint32_t b01, uint32_t b10, uint32_t b11, auto in_f16) {
        // entries 16 kb .. 16 kb + 15 of the head dimension
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          uint32_t a[4];
          const int row = 16 * r + (lane & 15), c = 2 * kb + (lane >> 4);
          ldsm(q_addr + (c / 8) * kRows * 128 + swizzled<128>(row, c & 7), a);
          if constexpr (decltype(in_f16)::value) {
            mma_f16(x[r][0], a, b00, b01);
            mma_f16(x[r][1], a, b10, b11);
          } else {
            mma(x[r][0], a, b00, b01);
            mma(x[r][1], a, b10, b11);
          }
        }
      };
      if constexpr (!kE4m3) {
#pragma unroll
        for (int kb = 0; kb < D / 16; ++kb) {
          uint32_t b[4];
          const int row = my_pos + (lane >> 4) * 8 + (lane & 7), c = 2 * kb + ((lane >> 3) & 1);
          ldsm(k_addr + (c / 8) * kTile * 128 + swizzled<128>(row, c & 7), b);
          dot16(kb, b[0], b[1], b[2], b[3], std::false_type{});
        }
      } else {
        auto dot32 = [&](int kb, auto in_f16) {
          uint32_t b[4];
          const int row = my_pos + (lane >> 4) * 8 + (lane & 7), c = 2 * kb + ((lane >> 3) & 1);
          ldsm(k_addr + swizzled<S::kPanelBytes>(row, c), b);
          uint32_t w[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (decltype(in_f16)::value) {
              w[i][0] = codes_f16(b[i]);
              w[i][1] = codes_f16(b[i] >> 16);
            } else {
              w[i][0] = widen(__byte_perm(b[i], 0, 0x1404));
              w[i][1] = widen(__byte_perm(b[i], 0, 0x3424));
            }
          }
          dot16(2 * kb, w[0][0], w[0][1], w[2][0], w[2][1], in_f16);
          dot16(2 * kb + 1, w[1][0], w[1][1], w[3][0], w[3][1], in_f16);
        };
        // (in f16 whatever Q is, and once more where it is bf16: with the two beside each other the
        // usual key tile takes 4% longer)
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) dot32(kb, std::true_type{});
        if (q_wide) {
#pragma unroll
          for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[r][n][i] = 0.f;
#pragma unroll 1
          for (int kb = 0; kb < D / 32; ++kb) dot32(kb, std::false_type{});
        }
      }
      // scores in units of log 2, and what a row does not see
      const bool whole = note.start >= seen_lo(p, note.L - 1) && note.start + kTile <= seen_hi(p, pos0, note.L);
      float k_scale[2][2];
      [[maybe_unused]] float v_scale[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        k_scale[n][0] = k_scale[n][1] = xscale;
        if constexpr (kE4m3) {
          const float2 f = *reinterpret_cast<const float2*>(&sm.scales[s][0][my_pos + 8 * n + j2]);
          const float2 v = *reinterpret_cast<const float2*>(&sm.scales[s][1][my_pos + 8 * n + j2]);
          k_scale[n][0] *= f.x;
          k_scale[n][1] *= f.y;
          v_scale[n][0] = v.x;
          v_scale[n][1] = v.y;
        }
      }
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          int lo = 0, hi = 0x7fffffff;
          if (!whole) {
            const int pos = pos0 + (16 * r + 8 * half + quad) / p.G;
            lo = seen_lo(p, pos) - note.start;
            hi = min(seen_hi(p, pos, note.L), note.L) - note.start;
          }
          float top = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float y = x[r][n][2 * half + i] * k_scale[n][i];
              const int at = my_pos + 8 * n + j2 + i;
              if (!whole && (at < lo || at >= hi)) y = -INFINITY;
              x[r][n][2 * half + i] = y;
              top = fmaxf(top, y);
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          if ((lane & 3) == 0) reinterpret_cast<float*>(&sm.top[16 * r + 8 * half + quad])[warp] = top;
        }
      // cold: a scale of a place that some row does not see may be anything (else the key tile's
      // are finite, and a weight of 0 stays 0), or P is bf16
      bool cold = v_wide || !v_whole;
      if (!compute_sync_and(ok && narrow)) {
        // (out of the way: a part's first scales, ones that do not fit or are not finite)
        if constexpr (kE4m3) {
          const uint32_t bits = scale_bits();
          const bool some = bits != 0, finite = bits < 0x7f800000u;
          int4 span;  // largest and smallest exponent; whether one does not fit, is not finite
          span.x = __reduce_max_sync(0xffffffffu, some && finite ? (int)(bits >> 23) : -1);
          span.y = __reduce_min_sync(0xffffffffu, some && finite ? (int)(bits >> 23) : 255);
          span.z = __any_sync(0xffffffffu, some && finite && !narrow);
          span.w = __any_sync(0xffffffffu, !finite);
          if (lane == 0) sm.span[warp] = span;
        }
        ok = compute_sync_and(ok);
        if (!ok) break;
        if constexpr (kE4m3) {
          int most = -1, least = 255;
          bool misfit = false;
#pragma unroll
          for (int w = 0; w < kComputeWarps; ++w) {
            const int4 span = sm.span[w];
            most = max(most, span.x);
            least = min(least, span.y);
            misfit |= span.z != 0;
            cold |= span.w != 0;
          }
          if (unit == kUnset) {
            if (most >= 0) {
              // (F and 1 / F are normal numbers, and what fits is finite)
              v_wide = most < 8 || most > 247 || least < most - kSpan;
              unit = v_wide ? 0 : (uint32_t)(most - kSpan) << 23;
              if (!v_wide) factor = __uint_as_float((254u << 23) - unit);
            }
          } else if (misfit) {  // from here on O and P are not scaled
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
              for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[r][n][i] *= __uint_as_float(unit);
            factor = 1.f;
            unit = 0;
            v_wide = true;
          }
          cold |= v_wide;
        }
      }
      if constexpr (kE4m3) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          v_scale[n][0] *= factor;
          v_scale[n][1] *= factor;
        }
      }
      // the second half of the key tile: the weights, then O
      auto weigh = [&](auto is_cold) {
        constexpr bool kCold = decltype(is_cold)::value;
        float keep[kR][2];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float4 t = sm.top[16 * r + 8 * half + quad];
            const float now = fmaxf(fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w)), m[r][half]);
            const float ref = now == -INFINITY ? 0.f : now;
            keep[r][half] = exp2_approx(m[r][half] - ref);
            moved |= now != m[r][half];
            m[r][half] = now;
            l[r][half] *= keep[r][half];
            const int row = 16 * r + 8 * half + quad;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float w0 = exp2_approx(x[r][n][2 * half] - ref), w1 = exp2_approx(x[r][n][2 * half + 1] - ref);
              l[r][half] += w0 + w1;
              float y0 = w0, y1 = w1;
              if constexpr (kE4m3) {
                y0 *= v_scale[n][0];
                y1 *= v_scale[n][1];
                if constexpr (kCold) {
                  // a weight of 0 stays 0 whatever the scale of a place that the row does not see
                  if (x[r][n][2 * half] == -INFINITY) y0 = 0.f;
                  if (x[r][n][2 * half + 1] == -INFINITY) y1 = 0.f;
                }
              }
              *reinterpret_cast<uint32_t*>(sm.pw + swizzled<128>(row, 2 * warp + n) + j2 * 2) =
                  kE4m3 && !(kCold && v_wide) ? pack_f16(y0, y1) : pack_bf16(y0, y1);
            }
          }
        compute_sync();
        // O: this warp's columns; the exponent's argument moves little, so most tiles keep
        // every maximum and skip the rescaling
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[r][n][i] *= keep[r][i >> 1];
        }
        // rows of V that no token of the request sees count as zeros
        auto v_mask = [&](int pos) {  // positions pos, pos + 1 of the tile, as a mask of two halves
          const int g = note.start + pos;
          return (g >= lo_all && g < note.L ? 0x0000ffffu : 0u) |
                 (g + 1 >= lo_all && g + 1 < note.L ? 0xffff0000u : 0u);
        };
        auto weigh16 = [&](int kb) {  // positions 16 kb .. 16 kb + 15
          uint32_t a[kR][4];
#pragma unroll
          for (int r = 0; r < kR; ++r)
            ldsm(p_addr + swizzled<128>(16 * r + (lane & 15), 2 * kb + (lane >> 4)), a[r]);
          const int row = 16 * kb + (lane & 15);
          if constexpr (!kE4m3) {
#pragma unroll
            for (int n = 0; n < kN; n += 2) {
              uint32_t b[4];
              const int c = warp * kN + n + (lane >> 4);
              ldsm_t(v_addr + (c / 8) * kTile * 128 + swizzled<128>(row, c & 7), b);
              if (!v_whole) {
                const uint32_t lo = v_mask(16 * kb + j2), hi = v_mask(16 * kb + 8 + j2);
                b[0] &= lo; b[1] &= hi; b[2] &= lo; b[3] &= hi;
              }
              if (!whole) {
                // A value that is not finite reaches the rows that see its position only:
                // it is taken out here and counted with the rows' visibility as weights.
                bool bad = false;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  bad |= (b[i] & 0x7f80u) == 0x7f80u || (b[i] & 0x7f800000u) == 0x7f800000u;
                if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
                  for (int kind = 0; kind < 3; ++kind) {  // +infinity, -infinity, not a number
                    uint32_t is[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      is[i] = 0;
#pragma unroll
                      for (int e = 0; e < 2; ++e) {
                        const uint32_t v = (b[i] >> (16 * e)) & 0xffffu;
                        const bool yes = kind == 0 ? v == 0x7f80u : kind == 1 ? v == 0xff80u : (v & 0x7fffu) > 0x7f80u;
                        if (yes) is[i] |= 0x3f80u << (16 * e);  // 1
                      }
                    }
                    const float add = kind == 0 ? INFINITY : kind == 1 ? -INFINITY : __uint_as_float(0x7fffffffu);
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                      uint32_t see[4];
#pragma unroll
                      for (int i = 0; i < 4; ++i) {
                        const int pos = pos0 + (16 * r + 8 * (i & 1) + quad) / p.G;
                        const int g = note.start + 16 * kb + 8 * (i >> 1) + j2;
                        const int lo = seen_lo(p, pos), hi = min(seen_hi(p, pos, note.L), note.L);
                        see[i] = (g >= lo && g < hi ? 0x3f80u : 0u) | (g + 1 >= lo && g + 1 < hi ? 0x3f800000u : 0u);
                      }
#pragma unroll
                      for (int e = 0; e < 2; ++e) {
                        float c4[4] = {0.f, 0.f, 0.f, 0.f};
                        mma(c4, see, is[2 * e], is[2 * e + 1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                          if (c4[i] > 0.f) o[r][n + e][i] += add;
                      }
                    }
                  }
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    if ((b[i] & 0x7f80u) == 0x7f80u) b[i] &= 0xffff0000u;
                    if ((b[i] & 0x7f800000u) == 0x7f800000u) b[i] &= 0x0000ffffu;
                  }
                }
              }
#pragma unroll
              for (int r = 0; r < kR; ++r) {
                mma(o[r][n], a[r], b[0], b[1]);
                mma(o[r][n + 1], a[r], b[2], b[3]);
              }
            }
          } else {
            // 16 columns per 16-byte chunk: the even ones, then the odd ones.  Codes in use have
            // no bad values (a bad row has a bad scale, which is in P of the rows that see it).
            constexpr int kChunks = D / kComputeWarps / 16;  // 2 (D = 128) or 1
            uint32_t b[4];
            const int c = warp * kChunks + (kChunks == 2 ? lane >> 4 : 0);
            ldsm_t(v_addr + swizzled<S::kPanelBytes>(row, c), b);
            if (!v_whole) {
              const uint32_t lo = v_mask(16 * kb + j2), hi = v_mask(16 * kb + 8 + j2);
              b[0] &= lo; b[1] &= hi; b[2] &= lo; b[3] &= hi;
            }
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
              if (kCold && v_wide) {
                const uint32_t e0 = widen(__byte_perm(b[2 * ch], 0, 0x2404)), d0 = widen(b[2 * ch]);
                const uint32_t e1 = widen(__byte_perm(b[2 * ch + 1], 0, 0x2404)), d1 = widen(b[2 * ch + 1]);
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                  mma(o[r][2 * ch], a[r], e0, e1);
                  mma(o[r][2 * ch + 1], a[r], d0, d1);
                }
                continue;
              }
              // columns of two positions: (0 1 | 0 1) to (0 | 0), (1 | 1)
              const uint32_t b0 = __byte_perm(b[2 * ch], 0, 0x3120), b1 = __byte_perm(b[2 * ch + 1], 0, 0x3120);
              const uint32_t e0 = codes_f16(b0), e1 = codes_f16(b1);
              const uint32_t d0 = codes_f16(b0 >> 16), d1 = codes_f16(b1 >> 16);
#pragma unroll
              for (int r = 0; r < kR; ++r) {
                mma_f16(o[r][2 * ch], a[r], e0, e1);
                mma_f16(o[r][2 * ch + 1], a[r], d0, d1);
              }
            }
          }
        };
        if constexpr (!kCold) {
#pragma unroll
          for (int kb = 0; kb < kTile / 16; ++kb) weigh16(kb);
        } else {
#pragma unroll 1
          for (int kb = 0; kb < kTile / 16; ++kb) weigh16(kb);
        }
      };
      if constexpr (!kE4m3) {
        weigh(std::false_type{});
      } else {
        if (!cold) weigh(std::false_type{});
        else weigh(std::true_type{});
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.empty[s]);
        if (note.flags & kLast) mbar_arrive(&sm.qempty[item & 1]);
      }
      if (!(note.flags & kLast)) continue;

      // ---- the end of this CTA's part of the item: the sums of the four warps' positions
      const bool done = (note.flags & kBegins) && (note.flags & kEnds);
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float t = l[r][half];
          t += __shfl_xor_sync(0xffffffffu, t, 1);
          t += __shfl_xor_sync(0xffffffffu, t, 2);
          if ((lane & 3) == 0) reinterpret_cast<float*>(&sm.top[16 * r + 8 * half + quad])[warp] = t;
        }
      compute_sync();
      const int place = (note.flags & kBegins) ? 1 : 0;
      const int rows = note.n * p.G;
      const float undo = factor == 1.f ? 1.f : __uint_as_float(unit);
      if (!done && place == 1 && tid == 0)
        pieces.notes[cta] = PieceNote{note.t0 * p.H + note.h * p.G, note.n, note.pieces, 0};
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = 16 * r + 8 * half + quad;
          const float4 t = sm.top[row];
          const float sum = (t.x + t.y) + (t.z + t.w);
          if (row >= rows) continue;
          const int tok = row / p.G;
          const size_t out_row = (size_t)(note.t0 + tok) * p.H + note.h * p.G + (row - tok * p.G);
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const size_t piece = ((size_t)cta * 2 + place) * kRows + row;
          if (warp == 0 && (lane & 3) == 0) {
            if (!done) pieces.ml[piece] = make_float2(m[r][half], sum);
            else if (p.lse) p.lse[out_row] = (m[r][half] + log2f(sum)) * kLn2;
          }
          if constexpr (!kE4m3) {
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              const int col = warp * (D / kComputeWarps) + 8 * n + j2;
              const float y0 = o[r][n][2 * half], y1 = o[r][n][2 * half + 1];
              if (done) *reinterpret_cast<uint32_t*>(p.out + out_row * D + col) = pack_bf16(y0 * inv, y1 * inv);
              else *reinterpret_cast<float2*>(pieces.o + piece * D + col) = make_float2(y0, y1);
            }
          } else {
#pragma unroll
            for (int n = 0; n < kN; n += 2) {  // even and odd columns: four in a row
              const int col = warp * (D / kComputeWarps) + 8 * n + 2 * j2;
              // (times 1 / l first where the row ends here: a sum of weights is 1 or more)
              const float by = done ? inv : 1.f;
              const float y0 = o[r][n][2 * half] * by * undo, y1 = o[r][n + 1][2 * half] * by * undo;
              const float y2 = o[r][n][2 * half + 1] * by * undo, y3 = o[r][n + 1][2 * half + 1] * by * undo;
              if (done)
                *reinterpret_cast<uint2*>(p.out + out_row * D + col) = make_uint2(pack_bf16(y0, y1), pack_bf16(y2, y3));
              else
                *reinterpret_cast<float4*>(pieces.o + piece * D + col) = make_float4(y0, y1, y2, y3);
            }
          }
        }
      compute_sync();  // the sums have been read: the next tile's maxima may come
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
  }
}

template <int D, int kRows, bool kE4m3>
cudaError_t launch_window(const AttentionArgs& a, cudaStream_t stream) {
  using Sm = Smem<D, kRows, kE4m3>;
  using S = Shape<D, kRows, kE4m3>;
  static_assert(S::kCtas * (sizeof(Sm) + 1024 + 1024) <= 228 * 1024, "the window CTAs fit an SM");
  static_assert(S::kStages >= 2, "the ring holds two key tiles");
  CUtensorMap maps[2];
  const uint64_t rows = (uint64_t)a.c.num_pages * a.c.HKV * a.c.page_size;
  for (int i = 0; i < 2; ++i)
    if (!make_map_2d(&maps[i], kE4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     S::kElem, i ? a.c.v : a.c.k, D, rows, S::kPanelBytes / S::kElem,
                     a.c.page_size < kTile ? a.c.page_size : kTile,
                     S::kPanelBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  const size_t smem = sizeof(Sm) + 1024;
  static SmemSet set;
  cudaError_t e = allow_smem(window_kernel<D, kRows, kE4m3>, smem, set);
  if (e != cudaSuccess) return e;
  const Pieces pieces = pieces_at(a.workspace, 152 * S::kCtas, kRows);
  e = launch(window_kernel<D, kRows, kE4m3>, dim3(152 * S::kCtas), dim3(kThreads), smem, stream, true,
             maps[0], maps[1], a, pieces);
  if (e != cudaSuccess) return e;
  return launch_join_pieces(a, pieces, kRows, 152 * S::kCtas, stream);
}

template <int D, bool kE4m3>
cudaError_t by_rows(const AttentionArgs& a, cudaStream_t stream) {
  if (window_rows(a.max_tokens, a.G) == 16 || a.window_rows == 16) return launch_window<D, 16, kE4m3>(a, stream);
  if constexpr (kE4m3) return launch_window<D, 32, kE4m3>(a, stream);
  return cudaErrorInvalidValue;  // its limit is 16 rows
}

}  // namespace

int window_rows(int max_tokens, int G) { return (long long)max_tokens * G <= 16 ? 16 : 32; }

cudaError_t launch_window_attention(const AttentionArgs& a, cudaStream_t stream) {
  if (a.c.D == 128)
    return a.c.e4m3 ? by_rows<128, true>(a, stream) : by_rows<128, false>(a, stream);
  return a.c.e4m3 ? by_rows<64, true>(a, stream) : by_rows<64, false>(a, stream);
}

}  // namespace kda
