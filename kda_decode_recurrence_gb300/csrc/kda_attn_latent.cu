// kda_attn_latent.cu -- attention of new tokens over a paged latent cache, absorbed form.
//
//   Every query head reads the same cached row r_j = (c_j, p_j) of 512 + 64 entries:
//     x_j = scale q . r_j,   o = sum e^(x_j - m) c_j / sum e^(x_j - m),   lse = m + ln sum
//   over the positions j that the token sees (all before it, all of its request, or all
//   cached ones and the nodes of a drafted tree that its mask names).
//
// A row is 1152 bytes and takes 2176 operations per query row: HBM bounds up to about
// 100 rows per cached row, the tensor cores more.  Query rows (token x head) of a request lie
// one behind the other, 128 to a row tile.  A cluster of two CTAs works on (request, row tile)
// items, key tiles of 128 positions, with products of the pair (cta_group::2, M = 128):
//   S = Q R^T     128 x 128, contraction 576; a CTA holds 64 of the rows and 64 of the keys
//   P = 2^(S - m) in bf16, by the CTA that owns the rows, into its shared memory
//   O += P C      128 x 512, twice N = 256; a CTA holds 256 columns of C, all 128 keys
// P is in bf16 because C is, and a product takes one type: 2^-8 of a weight at most, as the output's own
// rounding (errors against 64 bits 0.0017-0.0021, of outputs rounded once 0.0017).  P in two bf16 parts would
// double PV, half of the products.
// A single CTA cannot: 128 rows of O take the whole tensor memory, and of Q 144 KB.  In the
// pair a CTA has 64 rows of Q (72 KB), and O and two S take 384 of its 512 columns.
//
// Keys and values are streamed: their memory is given back as soon as their products are done.
// C comes twice (a CTA's keys for S, its columns for O): a pair's operands must lie at the same
// addresses in both CTAs, and a CTA's keys hold the columns of O in another place than its
// partner's.  The second copy comes from L2, into which rows are fetched two key tiles ahead.
//
// Items' key tiles are divided evenly over the pairs (the last item of a share may be
// unfinished: its pieces are joined by a second kernel).  O is rescaled only when a row's
// maximum has grown by more than 2^8.
//
// 128 tokens over 300-20000, 32 heads: 233-246 us by box, 5.5-5.8 TB/s of cache (on one box 239 beside 228 when warps
// without a live row go through the softmax); 64 over 1000-8000, 96 heads: 81-83 us, 4.3-4.4 TB/s.
// A key tile takes some 2900 cycles of a pair: 2176 of products, 150 of their issue, 570 of waits for copies,
// since the rings hold one key tile; an item's ends some 10000 (O through registers, 64 rows a CTA), a call's
// beginning 11000 and the join 7-10 us.  (76 x 6001 positions: tensor cores 60 % of active cycles, DRAM 69 %.)
// 32 windows of 1-8 over 200-6000, 64 heads, pages of 16: 70 us, the copies of smaller boxes in a tile's chain.
// Measured and left: copies in units of one key panel (296 us against 251 then), four more warps for half of
// the output (an item's ends 8000, a tile 100-200 more: 255 us against 250), kItemCost of 4 to 6.
#include <cuda.h>

#include "kda_attn.cuh"
#include "kda_latent.h"
#include "kda_launch.h"
#include "kda_tcgen05.cuh"
#include "kda_tmap.h"

namespace kda {
namespace {

constexpr int kPairs = 76;          // of CTAs, one CTA per SM
constexpr int kTile = 128;          // positions per key tile
constexpr int kHalf = 64;           // of them per CTA, and rows of a row tile per CTA
constexpr int kRows = 128;          // rows per row tile
constexpr int kPanels = kLatentRow / 64;
constexpr int kPanelBytes = kHalf * 128;
// A unit of keys is three panels (64 keys x 192 entries), one of values four (64 keys x this CTA's 256
// columns); the rings hold a key tile's.
constexpr int kKeyPanels = 3, kKeys = kPanels / kKeyPanels, kKeyBytes = kKeyPanels * kPanelBytes;
constexpr int kValuePanels = 4, kValues = 2, kValueBytes = kValuePanels * kPanelBytes;
// A unit in shared memory: panels of 64 rows (panel after panel of 128-byte rows), or, grouped, panels of 8 rows
// (8 rows of all its panels, then the next 8).  Grouped, a copy takes 8 rows of a whole unit, else a page's
// rows, one panel each unless they are 64: a key tile of pages of 16 takes 40 copies in place of 68, of 32
// 40 in place of 34, of 64 and more 40 in place of 5.  So only pages of 16 are grouped.
// (32 windows of 1-8 over 200-6000, pages of 16: 73.4 -> 69.3 us.)
template <bool kGrouped>
constexpr int kPanelAt = kGrouped ? 1024 : kPanelBytes;            // between a unit's panels
template <bool kGrouped>
constexpr int kKeyGroup = kGrouped ? kKeyPanels * 1024 : 1024;     // between its groups of 8 rows
template <bool kGrouped>
constexpr int kValueGroup = kGrouped ? kValuePanels * 1024 : 1024;
constexpr int kAhead = 2;           // key tiles that are fetched into L2 before their copies
constexpr int kNotes = 4;           // items whose notes are kept
constexpr int kItemCost = 3;        // what an item's beginning and end take, in key tiles
constexpr unsigned long long kPartLimitNs = 60 * kWaitLimitNs;  // limit of a wait for a whole part
constexpr float kGrow = 8.f;        // growth of a maximum (log 2) that rescales O
// Warps: 0-3 the softmax, 4 the products (of the pair's first CTA), 5 copies keys, 6 values, 7 finds the
// share's items, 8-11 load queries and pass on values.
constexpr int kMmaWarp = 4, kKeyWarp = 5, kCopyWarp = 6, kItemWarp = 7, kValueWarp = 8, kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kTmemCols = 512, kColO = 0, kColS = 256;

// One pair's part of an item; count 0: no more.
struct Part {
  int b, t0, n, L;
  int row0;       // of the row tile, among the request's n H rows
  int tile0, count;
  int end;        // positions that some row sees end before this
  int whole;      // key tiles that end at or before this position are seen by every row
  int flags;
  int pieces;     // pairs that share the item
};
constexpr int kBegins = 1, kEnds = 2;

struct Smem {
  unsigned char q[kPanels][kPanelBytes];    // this CTA's 64 rows, 1024-aligned, swizzled panels
  unsigned char key[kKeys][kKeyBytes];
  unsigned char value[kValues][kValueBytes];
  unsigned char p[2][kPanelBytes];          // 64 rows x 64 keys, twice
  Part part[kNotes];
  float red[2][2 * kHalf];
  int bad[kNotes];                          // item + 1: live entries of values were taken out of that item
  long long scan[2][kWarps];
  long long first_unit;                     // of the request that holds the share's first unit
  int first_request;
  Request first;                            // it
  uint32_t tmem;
  // this CTA's own (a key tile's last unit of keys has been read when S is there, its last of values when PV
  // is done)
  uint64_t key_empty[kKeys - 1], value_full[kValues], value_empty[kValues - 1];
  uint64_t part_full[kNotes], part_empty[kNotes];
  uint64_t s_full[2], o_done, q_empty, halves[2], done;
  // the first CTA's, arrived at by both (key_ready: by both CTAs' copies)
  uint64_t key_ready[kKeys], value_ready[kValues], q_ready, p_ready, o_free;
};

__device__ __forceinline__ Request load_request(const LatentArgs& p, int b, bool report) {
  Request r;
  r.t0 = fresh(p.cu + b);
  r.n = fresh(p.cu + b + 1) - r.t0;
  r.L = fresh(p.lens + b);
  const bool good = r.t0 >= 0 && r.n >= 0 && r.t0 + (long long)r.n <= p.T &&
                    (!p.mask || r.n <= 32ll * p.mask_words) && r.L >= 0 &&
                    r.L <= (long long)p.c.max_pages * p.c.page_size;
  if (!good) {
    if (report) raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
    r.n = 0;
  }
  return r;
}
__device__ __forceinline__ int row_tiles(const LatentArgs& p, const Request& r) {
  return (int)(((long long)r.n * p.H + kRows - 1) / kRows);
}
// Positions that some row of the tile sees end before this.
__device__ __forceinline__ int tile_end(const LatentArgs& p, const Request& r, int tile) {
  if (!p.causal) return r.L;
  const int last = (int)min((long long)r.n * p.H, (long long)(tile + 1) * kRows) - 1;
  return min(r.L, max(0, r.L - r.n + last / p.H + 1));
}
// An item's key tiles: at least one, since rows that see nothing are written too.
__device__ __forceinline__ int key_tiles(int end) { return max(1, (end + kTile - 1) / kTile); }
__device__ __forceinline__ int item_units(const LatentArgs& p, const Request& r, int tile) {
  return kItemCost + key_tiles(tile_end(p, r, tile));
}

// Units of the requests of a warp's lanes: by the lane where there are few row tiles, together
// where there are many.
__device__ __forceinline__ long long request_units(const LatentArgs& p, const Request& r, int lane) {
  const int tiles = row_tiles(p, r);
  if (!p.causal) return (long long)tiles * item_units(p, r, 0);
  const bool many = tiles > 8;
  long long sum = 0;
  if (!many)
    for (int t = 0; t < tiles; ++t) sum += item_units(p, r, t);
  for (unsigned left = __ballot_sync(0xffffffffu, many); left; left &= left - 1) {
    const int src = __ffs(left) - 1;
    Request x;
    x.t0 = __shfl_sync(0xffffffffu, r.t0, src);
    x.n = __shfl_sync(0xffffffffu, r.n, src);
    x.L = __shfl_sync(0xffffffffu, r.L, src);
    const int all = row_tiles(p, x);
    long long part = 0;
    for (int t = lane; t < all; t += 32) part += item_units(p, x, t);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == src) sum = part;
  }
  return sum;
}

// A bounded wait of a whole warp.  What the other CTA's arrivals stand for (a copy, P, an O that has been read)
// is in its own memory, complete or fenced for its tensor core, and released to the cluster by the arrival.
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity) {
  return wait_together<true>(smem_u32(bar), parity);
}

// The entries of x (eight bf16) that are not finite become zeros.
__device__ __forceinline__ uint4 finite(uint4 x) {
  auto keep = [](uint32_t v) {
    return ((v & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) & v | ((v & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u) & v;
  };
  return make_uint4(keep(x.x), keep(x.y), keep(x.z), keep(x.w));
}

// Adds the live entries of the latents that were taken out of an item's partly seen key tiles to columns
// col .. col + 31 of one row's output: the weight of each is found again from the query and the row in memory.
// (Rare: values that are not finite.)
__device__ __noinline__ void add_bad_latents(const LatentArgs& p, int b, int L, int n, int from, int to,
                                             const int32_t* words, const kda_bf16* q, float m, int col, float* o) {
  const int32_t* table = p.c.page_table + (size_t)b * p.c.max_pages;
  auto value = [](kda_bf16 x) { return __uint_as_float((uint32_t)x << 16); };
  for (int j = from; j < to; ++j) {
    if (words && !(tree_bits(words, p.mask_words, n, j - (L - n)) & 1)) continue;
    const int page = table[j / p.c.page_size];
    if (page < 0 || page >= p.c.num_pages) continue;
    const kda_bf16* row = p.c.rows + ((size_t)page * p.c.page_size + j % p.c.page_size) * kLatentRow;
    float w = -1.f;
    for (int d = 0; d < 32; ++d) {
      const kda_bf16 v = row[col + d];
      if ((v & 0x7f80u) != 0x7f80u) continue;
      if (w < 0.f) {
        float x = 0.f;
        for (int e = 0; e < kLatentRow; ++e) x = fmaf(value(q[e]), value(row[e]), x);
        w = exp2_approx(x * (p.scale * kLog2E) - m);
      }
      o[d] = fmaf(w, value(v), o[d]);
    }
  }
}

template <bool kGrouped>
__global__ void __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap key_map, const __grid_constant__ CUtensorMap value_map,
                  const __grid_constant__ LatentArgs p, const Pieces pieces) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (tid == 0) {
    for (int s = 0; s < kKeys; ++s) {
      if (s < kKeys - 1) mbar_init(&sm.key_empty[s], 1);
      mbar_init(&sm.key_ready[s], 1);
    }
    for (int s = 0; s < kValues; ++s) {
      mbar_init(&sm.value_full[s], 1);
      if (s < kValues - 1) mbar_init(&sm.value_empty[s], 1);
      mbar_init(&sm.value_ready[s], 8);
    }
    for (int s = 0; s < kNotes; ++s) {
      mbar_init(&sm.part_full[s], 1);
      mbar_init(&sm.part_empty[s], rank == 0 ? 11 : 10);  // warps that read notes
      sm.bad[s] = 0;
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.halves[s], 2);
    }
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.done, 1);
    mbar_init(&sm.q_ready, 8);
    mbar_init(&sm.p_ready, 8);
    mbar_init(&sm.o_free, 8);
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc_pair(&sm.tmem, kTmemCols);
  pdl_wait();
  pdl_trigger();

  // ---- this pair's share: a thread counts a request, in passes
  if (blockIdx.x == 0 && tid == 0 && (fresh(p.cu) != 0 || fresh(p.cu + p.B) != p.T))
    raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
  if (rank == 0 && tid == 0) pieces.notes[pair].tokens = 0;
  const int passes = (p.B + kThreads - 1) / kThreads;
  long long mine = 0, before = 0, units = 0;
  Request r{0, 0, 0};
  for (int i = 0; i < passes; ++i) {
    const int b = i * kThreads + tid;
    r = Request{0, 0, 0};
    if (b < p.B) r = load_request(p, b, blockIdx.x == 0);
    mine = request_units(p, r, lane);
    long long all;
    before = units + scan_before<kWarps>(mine, sm.scan[i & 1], all);
    units += all;
  }
  const int used = (int)min((long long)pairs, units);
  const long long u0 = pair < used ? share_begin(units, used, pair) : 0;
  const long long u1 = pair < used ? share_begin(units, used, pair + 1) : 0;
  for (int i = 0; i < passes && u1 > u0; ++i) {
    const int b = i * kThreads + tid;
    if (passes > 1) {  // counted again
      if (i == 0) units = 0;
      r = Request{0, 0, 0};
      if (b < p.B) r = load_request(p, b, false);
      mine = request_units(p, r, lane);
      long long all;
      __syncthreads();
      before = units + scan_before<kWarps>(mine, sm.scan[i & 1], all);
      units += all;
    }
    if (u0 >= before && u0 < before + mine) {
      sm.first_request = b;
      sm.first_unit = before;
      sm.first = r;
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // barriers and tensor memory of both CTAs are there
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  bool ok = true;

  auto read_part = [&](int item, Part& part) {
    ok = ok && wait_pair(&sm.part_full[item % kNotes], (item / kNotes) & 1);
    if (!ok) return false;
    part = sm.part[item % kNotes];
    return part.count > 0;
  };
  auto leave_part = [&](int item) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.part_empty[item % kNotes]);
  };

  if (warp == kItemWarp) {
    // ---- the share's items
    int item = 0;
    auto put_note = [&](const Part& part) {
      // (a part over a very long cache may take more than a second)
      if (item >= kNotes)
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.part_empty[item % kNotes], (item / kNotes - 1) & 1, kPartLimitNs));
      if (ok && lane == 0) {
        sm.part[item % kNotes] = part;
        mbar_arrive(&sm.part_full[item % kNotes]);
      }
      __syncwarp();
      ++item;
    };
    long long unit = 0;
    int b = 0, tile = 0, tiles = 0, base = 0;
    Request r{0, 0, 0}, held{0, 0, 0};  // held: request base + lane
    auto fetch = [&]() {
      base = b;
      held = Request{0, 0, 0};
      if (b + lane < p.B) held = load_request(p, b + lane, false);
    };
    auto take = [&]() {  // the first request from b on that has rows
      while (b < p.B) {
        if (b >= base + 32) fetch();
        const unsigned some = __ballot_sync(0xffffffffu, held.n > 0) & (0xffffffffu << (b - base));
        if (some) {
          const int src = __ffs(some) - 1;
          b = base + src;
          r.t0 = __shfl_sync(0xffffffffu, held.t0, src);
          r.n = __shfl_sync(0xffffffffu, held.n, src);
          r.L = __shfl_sync(0xffffffffu, held.L, src);
          tile = 0;
          tiles = row_tiles(p, r);
          return;
        }
        b = base + 32;
      }
    };
    if (u1 > u0) {
      b = sm.first_request;
      unit = sm.first_unit;
      r = sm.first;
      tiles = row_tiles(p, r);
      base = b - 32;  // (the requests after it are fetched when they are wanted)
      // the row tile that holds u0
      if (tiles == 1) {
        // it is the only one
      } else if (!p.causal) {
        const int each = item_units(p, r, 0);
        tile = (int)((u0 - unit) / each);
        unit += (long long)tile * each;
      } else {
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
    }
    while (u1 > u0 && unit < u1 && b < p.B && ok) {
      const int end = tile_end(p, r, tile), all = key_tiles(end);
      const int from = (int)max(0ll, u0 - unit - kItemCost), to = (int)min((long long)all, u1 - unit - kItemCost);
      if (to > from) {
        Part part;
        part.b = b;
        part.t0 = r.t0;
        part.n = r.n;
        part.L = r.L;
        part.row0 = tile * kRows;
        part.tile0 = from;
        part.count = to - from;
        part.end = end;
        const int pos0 = r.L - r.n, first = pos0 + part.row0 / p.H;
        part.whole = p.mask ? (first >= 0 ? pos0 : 0) : p.causal ? first + 1 : first >= 0 ? r.L : 0;
        part.flags = (from == 0 ? kBegins : 0) | (to == all ? kEnds : 0);
        part.pieces = to == all ? 1 : share_of(units, used, unit + kItemCost + all - 1) - pair + 1;
        put_note(part);
      }
      unit += kItemCost + all;
      if (++tile >= tiles) {
        ++b;
        take();
      }
    }
    if (ok) put_note(Part{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0});
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
  } else if (warp == kKeyWarp || warp == kCopyWarp) {
    // ---- keys or values into their ring.  (This chain is as long as a key tile takes: no division in it.)
    const int page_shift = 31 - __clz(p.c.page_size), in_page = p.c.page_size - 1;
    const int box_shift = kGrouped ? 3 : min(page_shift, 6), rows_per_box = 1 << box_shift;
    const int half_boxes = kHalf >> box_shift, boxes = 2 * half_boxes;  // of a half, of a key tile
    const int nowhere = p.c.num_pages << page_shift;                    // a row past the end: zeros
    // a unit's copies, by lane: all panels of 64 rows at once, or of fewer rows a panel each
    const bool keys = warp == kKeyWarp;
    const int in = lane & (half_boxes - 1), panel = lane / half_boxes;
    const int panels = keys ? kKeyPanels : kValuePanels;
    const int copies = kGrouped || half_boxes == 1 ? 1 : panels;
    const uint32_t to = panel * kPanelBytes + in * rows_per_box * 128 * (kGrouped ? panels : 1);
    const uint32_t ready0 = cluster_addr(&sm.key_ready[0], 0);
    int tasks = 0, put = 0;      // key tiles, units so far
    int soon = -1, soon_in = 0;  // page and position in it to be fetched into L2 next, by lane
    Part part;
    for (int item = 0; read_part(item, part); leave_part(item), ++item) {
      const int32_t* table = p.c.page_table + (size_t)part.b * p.c.max_pages;
      const int first = part.tile0 * kTile, last = min(part.end, (part.tile0 + part.count) * kTile);
      int page = -1;  // of the 32 boxes under way, by lane
      // row of the cache where `box` (per lane) of the part's key tile i starts; past the end: zeros
      auto cache_row = [&](int i, int box) {
        const int at = i * boxes + box, pos = first + (at << box_shift);
        const int pg = __shfl_sync(0xffffffffu, page, at & 31);
        return pg >= 0 ? (pg << page_shift) + (pos & in_page) : nowhere;
      };
      // Rows of a later key tile (this part's, or the next one's where its note is there) are fetched into
      // L2: copies wait for room in the rings, which a key tile fills, and HBM is further away than that.
      // A tile's page is looked up one tile before it is needed.
      auto fetch_ahead = [&](int i) {
        if (soon >= 0 && soon < p.c.num_pages)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                           p.c.rows + (((size_t)soon << page_shift) + soon_in) * kLatentRow),
                       "r"(rows_per_box * kLatentRow * 2)
                       : "memory");
        soon = -1;
        const int at = i + kAhead;
        int pos = first + at * kTile + rank * kHalf + (lane << box_shift);
        const int32_t* of = table;
        bool some = pos < last;
        if (at >= part.count) {
          if (!__all_sync(0xffffffffu, mbar_test(smem_u32(&sm.part_full[(item + 1) % kNotes]), ((item + 1) / kNotes) & 1)))
            return;
          const Part& next = sm.part[(item + 1) % kNotes];
          pos += (next.tile0 - part.tile0 - part.count) * kTile;
          some = at - part.count < next.count && pos < next.end;
          of = p.c.page_table + (size_t)next.b * p.c.max_pages;
        }
        if (some && lane < half_boxes) {
          soon = fresh(of + (pos >> page_shift));
          soon_in = pos & in_page;
        }
      };
      for (int i = 0; i < part.count && ok; ++i, ++tasks) {
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
        if (keys) {
          // this CTA's half of the keys, three panels at a time; both CTAs' copies arrive at the first's barrier
          const int row = cache_row(i, rank * half_boxes + in);
#pragma unroll
          for (int k = 0; k < kKeys; ++k) {
            if (tasks > 0 && ok)  // the key tile before has been read
              ok = k < kKeys - 1 ? wait_pair(&sm.key_empty[k], (tasks - 1) & 1)
                                 : wait_pair(&sm.s_full[(tasks - 1) & 1], ((tasks - 1) >> 1) & 1);
            if (!ok) break;
            if (rank == 0 && lane == 0) mbar_expect_tx(&sm.key_ready[k], 2 * kKeyBytes);
            __syncwarp();
            if (panel < copies)
              tma_load_3d_pair(sm.key[k] + to, &key_map, ready0 + 8 * k, 0, row, k * kKeyPanels + panel);
            put = tasks * kKeys + k + 1;
          }
          fetch_ahead(i);
        } else {
          // this CTA's columns, half of the keys at a time
          const int row_lo = cache_row(i, in), row_hi = cache_row(i, half_boxes + in);
#pragma unroll
          for (int v = 0; v < kValues; ++v) {
            if (tasks > 0 && ok) ok = wait_pair(v < kValues - 1 ? &sm.value_empty[v] : &sm.o_done, (tasks - 1) & 1);
            if (!ok) break;
            if (lane == 0) mbar_expect_tx(&sm.value_full[v], kValueBytes);
            __syncwarp();
            if (panel < copies)
              tma_load_3d(sm.value[v] + to, &value_map, &sm.value_full[v], 0, v ? row_hi : row_lo,
                          rank * kValuePanels + panel);
            put = tasks * kValues + v + 1;
          }
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
    // Every copy lands before the CTA's memory is released, also when a wait gave up (keys: the first CTA
    // waits for both).
    if (!keys)
      for (int u = max(0, put - kValues); u < put; ++u) mbar_wait(&sm.value_full[u % kValues], (u / kValues) & 1);
    else if (rank == 0)
      for (int u = max(0, put - kKeys); u < put; ++u) mbar_wait(&sm.key_ready[u % kKeys], (u / kKeys) & 1);
  } else if (warp == kMmaWarp && rank == 0) {
    // ---- the products.  (The second CTA's warp would run ahead of the notes, and wait for a long part's end.)
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t q0 = smem_u32(sm.q[0]), key0 = smem_u32(sm.key[0]), value0 = smem_u32(sm.value[0]),
                   p0 = smem_u32(sm.p[0]);
    const uint32_t idesc_s = idesc_bf16(kTile, kRows, false, false), idesc_o = idesc_bf16(256, kRows, false, true);
    const uint32_t one = elect_one() ? 1u : 0u;
    int task = 0;  // key tiles so far
    Part part;
    for (int item = 0; read_part(item, part); leave_part(item), ++item) {
      const int count = __shfl_sync(0xffffffffu, part.count, 0);
      ok = wait_pair(&sm.q_ready, item & 1);
      for (int i = 0; i <= count && ok; ++i) {
        if (i < count) {
          const uint32_t s_col = base + kColS + (uint32_t)((task + i) & 1) * kHalf;
#pragma unroll 1
          for (int k = 0; k < kKeys && ok; ++k) {
            ok = wait_pair(&sm.key_ready[k], (task + i) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = smem_desc_sw128(q0 + k * kKeyBytes, 16, 1024);
            const uint64_t b = smem_desc_sw128(key0 + k * kKeyBytes, 16, kKeyGroup<kGrouped>);
#pragma unroll
            for (int j = 0; j < 4 * kKeyPanels; ++j) {  // 32 bytes on, or the next panel
              mma_bf16_pair_if(one, s_col, a + (j & 3) * 2 + (j >> 2) * (kPanelBytes / 16),
                               b + (j & 3) * 2 + (j >> 2) * (kPanelAt<kGrouped> / 16), idesc_s, k + j > 0 ? 1u : 0u);
            }
            mma_commit_pair_if(one, k < kKeys - 1 ? &sm.key_empty[k] : &sm.s_full[(task + i) & 1]);
          }
          if (i == count - 1) mma_commit_pair_if(one, &sm.q_empty);
        }
        if (i > 0 && ok) {
          const int g = task + i - 1;
          if (i == 1 && item > 0) ok = wait_pair(&sm.o_free, (item - 1) & 1);
          ok = ok && wait_pair(&sm.p_ready, g & 1);
#pragma unroll 1
          for (int v = 0; v < kValues && ok; ++v) {
            ok = wait_pair(&sm.value_ready[v], g & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = smem_desc_sw128(p0 + v * kPanelBytes, 16, 1024);
            const uint64_t c = smem_desc_sw128(value0 + v * kValueBytes, kPanelAt<kGrouped>, kValueGroup<kGrouped>);
#pragma unroll
            for (int j = 0; j < 8; ++j)  // 16 keys, then this CTA's next 128 columns
              mma_bf16_pair_if(one, base + kColO + (j >> 2) * 128, a + 2 * (j & 3),
                               c + (j & 3) * (2 * kValueGroup<kGrouped> / 16) + (j >> 2) * (2 * kPanelAt<kGrouped> / 16), idesc_o,
                               i > 1 || v > 0 || (j & 3) > 0 ? 1u : 0u);
            mma_commit_pair_if(one, v < kValues - 1 ? &sm.value_empty[v] : &sm.o_done);
          }
        }
      }
      task += count;
      if (!ok) break;
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
    mma_commit_pair_if(one, &sm.done);  // arrives when every product issued has completed
    mbar_wait(&sm.done, 0);
  } else if (warp >= kValueWarp) {
    // ---- each item's queries; values that have arrived, without the entries that some row must not see
    const int wv = warp - kValueWarp;
    int values = 0;
    Part part;
    for (int item = 0; read_part(item, part); leave_part(item), ++item) {
      // A warp takes 16 rows of the 64, 72 chunks each; lanes find a row's place each.
      const int first = part.row0 + rank * kHalf + wv * 16;
      const int live = (int)max(0ll, min(16ll, (long long)part.n * p.H - first));
      const int token = (first + lane) / p.H;
      const kda_bf16* mine = p.q;
      if (lane < live) {
        mine += (part.t0 + token) * p.q_stride + (size_t)(first + lane - token * p.H) * kLatentRow;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(mine), "r"(kLatentRow * 2) : "memory");
      }
      if (item > 0) ok = wait_pair(&sm.q_empty, (item - 1) & 1);
      if (!ok) break;
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int row = wv * 16 + i;
        const kda_bf16* src = reinterpret_cast<const kda_bf16*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), i));
        const uint32_t to = smem_u32(sm.q[lane >> 3] + swizzled<128>(row, lane & 7));
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (k < 2 || lane < 8)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + k * 4 * kPanelBytes),
                         "l"(src + (k * 32 + lane) * 8), "r"(i < live ? 16 : 0)
                         : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&sm.q_ready, 0));
      for (int i = 0; i < part.count && ok; ++i) {
        const int start = (part.tile0 + i) * kTile;
#pragma unroll 1
        for (int v = 0; v < kValues && ok; ++v, ++values) {
          const int s = values % kValues;
          ok = wait_pair(&sm.value_full[s], (values / kValues) & 1);
          if (!ok) break;
          if (start + kTile > part.whole) {
            // A quarter of the unit's 64 keys, four panels of eight chunks each.  0 x NaN would reach
            // rows that do not see it; those that do add it at the item's end.
            bool bad = false;
#pragma unroll 8
            for (int k = 0; k < 16; ++k) {
              const int n = k * 32 + lane, key = wv * 16 + ((n >> 3) & 15);
              uint4* x = reinterpret_cast<uint4*>(sm.value[s] + (n >> 7) * kPanelAt<kGrouped> + (key >> 3) * kValueGroup<kGrouped> +
                                                  swizzled<128>(key & 7, n & 7));
              const uint4 y = *x;
              const bool live = start + v * kHalf + key < part.L;
              const uint4 z = live ? finite(y) : make_uint4(0, 0, 0, 0);
              if (y.x != z.x || y.y != z.y || y.z != z.z || y.w != z.w) {
                *x = z;
                bad |= live;
              }
            }
            if (__any_sync(0xffffffffu, bad)) {  // for the rows of both CTAs
              if (lane == 0)
                for (int to = 0; to < 2; ++to)
                  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&sm.bad[item % kNotes], to)),
                               "r"(item + 1)
                               : "memory");
              asm volatile("fence.acq_rel.cluster;" ::: "memory");
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(&sm.value_ready[s], 0));
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
  } else if (warp < 4) {
    // ---- the softmax: thread (row, half of the keys)
    const int row = tid & (kHalf - 1), half = tid >> 6;
    const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
    const float c = p.scale * kLog2E;
    const float2 c2 = make_float2(c, c);
    const uint32_t p_ready = cluster_addr(&sm.p_ready, 0), o_free = cluster_addr(&sm.o_free, 0);
    unsigned char* const p_row = sm.p[half];
    int task = 0, swaps = 0;
    // The partner's value: the other half of this row's keys.
    auto swap = [&](float x) {
      sm.red[swaps & 1][tid] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.halves[warp & 1]);
      ok = ok && wait_pair(&sm.halves[warp & 1], swaps & 1);
      const float y = sm.red[swaps & 1][tid ^ kHalf];
      ++swaps;
      return y;
    };
    Part part;
    for (int item = 0; read_part(item, part); leave_part(item), ++item) {
      const int L = part.L, n = part.n;
      const int in = rank * kHalf + row, flat = part.row0 + in;
      const int token = flat / p.H, pos = L - n + token;
      const bool live = flat < (long long)n * p.H;
      const bool idle = !__any_sync(0xffffffffu, live);  // (what is left in P stays in rows that nobody reads)
      const int row_hi = pos < 0 || !live ? 0 : p.causal ? min(pos + 1, L) : L;
      const int32_t* words = p.mask && live ? p.mask + (size_t)(part.t0 + token) * p.mask_words : nullptr;
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int i = 0; i < part.count; ++i, ++task) {
        ok = wait_pair(&sm.s_full[task & 1], (task >> 1) & 1);
        if (!ok) break;
        if (idle) {
          if (task > 0) ok = wait_pair(&sm.o_done, (task - 1) & 1);  // (no word twice of one product)
          if (!ok) break;
          if (lane == 0) mbar_arrive_cluster(p_ready);
          continue;
        }
        tc_fence_after();
        const int start = (part.tile0 + i) * kTile + half * kHalf;
        float x[2][32];
        const uint32_t s_col = lanes + kColS + (uint32_t)(task & 1) * kHalf;
        tmem_ld_32cols(s_col, x[0]);
        tmem_ld_32cols(s_col + 32, x[1]);
        tmem_ld_wait();
        const bool whole = (part.tile0 + i + 1) * kTile <= part.whole;
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 a = __fmul2_rn(make_float2(x[h][e], x[h][e + 1]), c2);
            x[h][e] = a.x;
            x[h][e + 1] = a.y;
          }
          if (!whole) {
            const int at = start + 32 * h;
            uint32_t see = columns(0, row_hi - at);
            if (words && row_hi > 0) see &= tree_bits(words, p.mask_words, n, at - (L - n));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1)) x[h][e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) top = max3(top, x[h][e], x[h][e + 1]);
        }
        const float now = max3(m, top, swap(top));
        if (task > 0) ok = ok && wait_pair(&sm.o_done, (task - 1) & 1);  // O and P are at rest
        if (!ok) break;
        // (both warps of a row decide alike: they have the same rows, maxima and so references)
        if (__any_sync(0xffffffffu, live && now > m + kGrow)) {  // (a row that is not live may hold anything)
          const float keep = exp2_approx(m - (now == -INFINITY ? 0.f : now));
          l2.x *= keep;
          l2.y *= keep;
          if (i > 0) {
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < 256; cc += 16) {
              float o[16];
              tmem_ld_16cols(lanes + kColO + cc, o);
              tmem_ld_wait();
              uint32_t ob[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) ob[e] = __float_as_uint(o[e] * keep);
              tmem_st_16cols(lanes + kColO + cc, ob);
            }
            tmem_st_wait();
          }
          m = now;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const float2 nref = make_float2(-ref, -ref);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              const float2 y = __fadd2_rn(make_float2(x[h][e + k], x[h][e + k + 1]), nref);
              const float2 v = make_float2(exp2_approx(y.x), exp2_approx(y.y));
              l2 = __fadd2_rn(l2, v);
              w[k / 2] = pack_bf16(v.x, v.y);
            }
            *reinterpret_cast<uint4*>(p_row + swizzled<128>(row, 4 * h + e / 8)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_ready);
      }
      if (!ok) break;
      if (idle) {
        ok = wait_pair(&sm.o_done, (task - 1) & 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_cluster(o_free);
        continue;
      }
      const float l_half = l2.x + l2.y, l = l_half + swap(l_half);
      ok = ok && wait_pair(&sm.o_done, (task - 1) & 1);
      if (!ok) break;
      // ---- the end of this pair's part of the item
      tc_fence_after();
      const bool done = (part.flags & (kBegins | kEnds)) == (kBegins | kEnds);
      const size_t out_row = (size_t)part.t0 * p.H + flat;
      const size_t piece = ((size_t)pair * 2 + (part.flags & kBegins ? 1 : 0)) * kRows + in;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool bad = sm.bad[item % kNotes] == item + 1;
      if (live && half == 0) {
        if (!done) pieces.ml[piece] = make_float2(m, l);
        else if (p.lse) p.lse[out_row] = (m + log2f(l)) * kLn2;
      }
      if (rank == 0 && tid == 0 && (part.flags & (kBegins | kEnds)) == kBegins)
        pieces.notes[pair] = PieceNote{part.t0 * p.H + part.row0,
                                       (int)min((long long)kRows, (long long)n * p.H - part.row0), part.pieces, 0};
      int to_rows[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) to_rows[e] = __shfl_sync(0xffffffffu, live ? (int)out_row : -1, (lane & ~3) + e);
#pragma unroll 1
      for (int cc = 0; cc < 256; cc += 32) {
        float o[32];
        tmem_ld_32cols(lanes + kColO + cc, o);
        tmem_ld_wait();
        const int col = half * 256 + cc;
        if (bad && live) {
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = o[e];
          add_bad_latents(p, part.b, L, n, max(part.tile0, part.whole / kTile) * kTile,
                          min(row_hi, (part.tile0 + part.count) * kTile), words,
                          p.q + (part.t0 + token) * p.q_stride + (size_t)(flat - token * p.H) * kLatentRow,
                          m == -INFINITY ? 0.f : m, col, y);
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
              *reinterpret_cast<uint4*>(p.out + (size_t)to_rows[e] * kLatent + col + 8 * (lane & 3)) = y[e];
        } else if (live) {
          // [64 quarters of a half row][2 CTAs][128 threads]: the lanes of a warp write 512 bytes together
          float4* to = reinterpret_cast<float4*>(pieces.o + (piece - in) * kLatent) + (cc / 4 * 2 + rank) * 128 + tid;
#pragma unroll
          for (int e = 0; e < 32; e += 4) to[e / 4 * 256] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        __syncwarp();  // the next load is the whole warp's
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(o_free);
    }
    if (!ok && lane == 0) raise_status(p.dev_status, KDA_DEV_TIMEOUT);
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
// CTA (c, y) takes 16 columns from 16 (y / 2) on of either half of the 64 rows of the pair's CTA y % 2 in
// the item that pair c began: thread (row, half) as in the softmax.
constexpr int kJoinY = 32;
__global__ void __launch_bounds__(128) latent_join_kernel(const LatentArgs p, const Pieces s) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, rank = blockIdx.y & 1, cc = blockIdx.y >> 1;
  const PieceNote note = s.notes[c];
  const int row = rank * kHalf + (threadIdx.x & (kHalf - 1));
  if (row >= note.tokens) return;
  auto at = [&](int i) { return ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * kRows; };
  float m = -INFINITY, l = 0.f;
  float4 o[4] = {};
#pragma unroll 2
  for (int i = 0; i < note.pieces; ++i) {
    const float2 ml = s.ml[at(i) + row];
    const float4* from = reinterpret_cast<const float4*>(s.o + at(i) * kLatent) + (cc * 8 + rank) * 128 + threadIdx.x;
    float4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = from[e * 256];
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
  const size_t out_row = (size_t)note.row0 + row;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint4* to = reinterpret_cast<uint4*>(p.out + out_row * kLatent + (threadIdx.x >= kHalf ? kLatent / 2 : 0) + 16 * cc);
#pragma unroll
  for (int e = 0; e < 4; e += 2)
    to[e / 2] = make_uint4(pack_bf16(o[e].x * inv, o[e].y * inv), pack_bf16(o[e].z * inv, o[e].w * inv),
                           pack_bf16(o[e + 1].x * inv, o[e + 1].y * inv), pack_bf16(o[e + 1].z * inv, o[e + 1].w * inv));
  if (p.lse && cc == 0 && threadIdx.x < kHalf) p.lse[out_row] = (m + log2f(l)) * kLn2;
}

template <bool kGrouped>
cudaError_t launch_latent(const LatentArgs& a, cudaStream_t stream) {
  static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "a CTA fits an SM");
  // The cache as [panel of 64 entries][row][64 entries]: a box of several panels lands as a unit's layout.
  const uint32_t page_rows = a.c.page_size < kHalf ? a.c.page_size : kHalf;
  const bool whole_unit = kGrouped || page_rows == kHalf;
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i)
    if (!make_map_3d_bf16(&maps[i], a.c.rows, 64, (uint64_t)a.c.num_pages * a.c.page_size, kPanels, kLatentRow * 2, 128,
                          64, kGrouped ? 8 : page_rows, whole_unit ? (i ? kValuePanels : kKeyPanels) : 1))
      return cudaErrorInvalidValue;
  const size_t smem = sizeof(Smem) + 1024;
  static SmemSet set;
  cudaError_t e = allow_smem(latent_kernel<kGrouped>, smem, set);
  if (e != cudaSuccess) return e;
  const Pieces pieces = pieces_at(a.workspace, kPairs, kRows);
  e = launch_pairs(latent_kernel<kGrouped>, dim3(2 * kPairs), dim3(kThreads), smem, stream, maps[0], maps[1], a, pieces);
  if (e != cudaSuccess) return e;
  return launch(latent_join_kernel, dim3(kPairs, kJoinY), dim3(128), 0, stream, true, a, pieces);
}

}  // namespace

size_t latent_workspace_bytes(int B, int T, int H) {
  if (B < 0 || T < 0 || H < 1) return 0;
  return (pieces_bytes(kPairs, kRows, kLatent) + 255) & ~(size_t)255;
}

cudaError_t launch_latent_attention(const LatentArgs& a, cudaStream_t stream) {
  return a.c.page_size == 16 ? launch_latent<true>(a, stream) : launch_latent<false>(a, stream);
}

}  // namespace kda
