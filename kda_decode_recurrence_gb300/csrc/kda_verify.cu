// kda_verify.cu -- verification of drafted tokens from given uniform numbers.
//
//   draft i of a request is accepted iff all before it were and
//   u_i q_i(x_i) < p_i(x_i) (the product and the comparison exact in fp64);
//   with j accepted, one token is drawn from the weights
//     w = max(p_j - q_j, 0) after a rejection,  w = p_n after n acceptances:
//   the smallest v with C(v) > u C(V - 1), C the running sum of w.
//
// A draw reads two rows of V probabilities (one if all drafts were accepted) and
// does about 13 operations per entry: HBM bounds it.  fp64 adds cannot keep
// up (152 SMs x 2 per clock = 0.6 T/s against 0.8 T entries/s from HBM), so
// sums are pairs of fp32 (hi + lo) for up to 32 entries of a lane, pairs of those for up to 16
// such runs, and fp64 beyond that and where warps are joined: neighbours in a large vocabulary
// lie 1e-6 of the sum apart.
// A pair's low part takes a rounded addition per entry, so that after n of them it is off by
// at most (n^2 / 2 + 3.5 n) 2^-48 of the sum: 2^-38.7 for 32, 2^-40.5 for the 16 runs (measured
// on weights that span many octaves: 2^-48; with one pair for all 2^-45 after 128 entries,
// 2^-34 after 16384).
//
// A cluster of CTAs serves a request, its warps a segment of the row each; the
// segments' sums meet through distributed shared memory, so that one launch does
// it all.  The cluster has as many CTAs (8, 4, 2 or 1) as let all requests run at
// once: a second wave would find few CTAs left to keep HBM busy.
//
// 256 requests of 1 .. 7 drafts over 131072 tokens: 268 MB in 56 us, 4.8 TB/s (a copy:
// 6.7); point drafts 134 MB in 47.  Loads are waited for (8.7 of 16 cycles per instruction),
// barriers 2.5, issue is at 42% and the SMs are busy for 80% of the time: the chain before a
// request's first row (offsets, drafted token, two probabilities) and the cluster's two
// barriers after its last have nothing beside them, all requests being in one wave.
// Four over 32001: 12.5 us with the host's call.  800 over 131072, four runs of 32 entries per
// lane: 247 us (one pair for all 128: 234).
#include <cooperative_groups.h>

#include <type_traits>

#include "kda_common.cuh"
#include "kda_paged.h"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;               // CTAs per request
constexpr int kCtasPerSm = 16;
constexpr int kSms = 152;
constexpr int kBlocks = 8;                   // blocks a segment is searched by
constexpr int kRun = 32;                     // entries that a lane adds in one pair,
constexpr int kRuns = 16;                    // and such pairs in one more

struct Pair {
  float hi, lo;
};

// s += d + e with the rounding error of hi kept in lo (Knuth's two-sum).
__device__ __forceinline__ void add(Pair& s, float d, float e) {
  const float t = s.hi + d;
  const float b = t - s.hi;
  s.lo += ((s.hi - (t - b)) + (d - b)) + e;
  s.hi = t;
}

__device__ __forceinline__ double warp_total(Pair s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, s.hi, o), lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
    add(s, hi, lo);
  }
  return (double)s.hi + (double)s.lo;
}

__device__ __forceinline__ double warp_total(double s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ double warp_scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The weights of one draw.
struct Weights {
  const float* p;
  const float* q;  // null: nothing is taken off
  int skip;        // entry whose draft probability is 1 (point drafts), or -1

  // w_v = hi + lo exactly (0 where not positive or not a number).
  __device__ __forceinline__ void get(float pv, float qv, int v, float& hi, float& lo) const {
    const float d = pv - qv;
    const bool some = pv > qv && v != skip;
    hi = some ? d : 0.f;
    lo = some ? (pv - d) - qv : 0.f;  // exact for p > q >= 0 (Dekker)
  }
  __device__ __forceinline__ void load(int v, float& hi, float& lo) const {
    get(__ldg(p + v), q ? __ldg(q + v) : 0.f, v, hi, lo);
  }
};

// This lane's share of the weights lo..hi-1 (both multiples of 4, or hi = V): by
// 16-byte loads where the rows allow it (kVec), else one entry at a time.
template <bool kHasQ, bool kVec>
__device__ __forceinline__ Pair lane_sum(const Weights& w, int lo, int hi, int lane) {
  constexpr int kEach = kVec ? 4 : 1;
  constexpr int kUnroll = kVec ? 2 : 4;
  constexpr int kStep = 32 * kEach;
  Pair s = {0.f, 0.f};
  int v = lo + lane * kEach;
  for (; v + kStep * (kUnroll - 1) + kEach <= hi; v += kStep * kUnroll) {
    float pv[kUnroll * kEach], qv[kUnroll * kEach];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if constexpr (kVec) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(w.p + v + kStep * i));
        pv[4 * i] = x.x; pv[4 * i + 1] = x.y; pv[4 * i + 2] = x.z; pv[4 * i + 3] = x.w;
      } else {
        pv[i] = __ldg(w.p + v + kStep * i);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if constexpr (kHasQ && kVec) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(w.q + v + kStep * i));
        qv[4 * i] = x.x; qv[4 * i + 1] = x.y; qv[4 * i + 2] = x.z; qv[4 * i + 3] = x.w;
      } else if constexpr (kVec) {
        qv[4 * i] = qv[4 * i + 1] = qv[4 * i + 2] = qv[4 * i + 3] = 0.f;
      } else {
        qv[i] = kHasQ ? __ldg(w.q + v + kStep * i) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll * kEach; ++i) {
      float d, e;
      w.get(pv[i], qv[i], v + kStep * (i / kEach) + i % kEach, d, e);
      add(s, d, e);
    }
  }
  for (; v < hi; v += kStep)
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (v + i >= hi) break;
      float d, e;
      w.get(__ldg(w.p + v + i), kHasQ ? __ldg(w.q + v + i) : 0.f, v + i, d, e);
      add(s, d, e);
    }
  return s;
}
template <bool kVec>
__device__ __forceinline__ Pair lane_sum(const Weights& w, int lo, int hi, int lane) {
  return w.q ? lane_sum<true, kVec>(w, lo, hi, lane) : lane_sum<false, kVec>(w, lo, hi, lane);
}

// The first lane with a weight x whose inclusive running sum c passes `target`;
// if rounding lets none pass, the last lane with a weight (0: no weight at all).
__device__ __forceinline__ int first_past(double c, double x, double target) {
  const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
  const unsigned past = __ballot_sync(0xffffffffu, c > target) & some;
  return past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
}

// The entries of a block of a warp's segment.
__host__ __device__ __forceinline__ int segment_of(int V, int segments) { return ((V + segments - 1) / segments + 3) & ~3; }
__host__ __device__ __forceinline__ int block_of(int segment) { return ((segment + kBlocks - 1) / kBlocks + 127) & ~127; }

// kLong: a lane has more than kRun entries of a block.
template <bool kVec, bool kLong>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) verify_kernel(const VerifyArgs a, const int size) {
  __shared__ int s_taken, s_found;
  using Sum = std::conditional_t<kLong, double, Pair>;
  __shared__ Sum s_lane[kBlocks][kThreads];  // every lane's sum of each block of its segment
  __shared__ double s_own[kWarps], s_base, s_target;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int segments = kWarps * size;  // of a row, one per warp
  const int b = blockIdx.x / size;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int d0 = a.cu[b], d1 = a.cu[b + 1];
  // The whole cluster sees the same range and leaves together.
  if (b == 0 && rank == 0 && tid == 0 && (a.cu[0] != 0 || a.cu[a.B] != a.N))
    raise_status(a.dev_status, KDA_DEV_BAD_SEQLEN);
  if (d0 < 0 || d1 < d0 || d1 > a.N) {
    if (rank == 0 && tid == 0) raise_status(a.dev_status, KDA_DEV_BAD_SEQLEN);
    return;
  }
  const int n = d1 - d0;
  const size_t row0 = (size_t)d0 + b;  // the request's first target row and output place

  // ---- how many drafts are accepted (warp 0 of every CTA, 32 at a time)
  if (warp == 0) {
    int taken = n;
    for (int i0 = 0; i0 < n && taken == n; i0 += 32) {
      const int i = i0 + lane;
      bool yes = true;
      if (i < n) {
        const int x = a.draft_tokens[d0 + i];
        yes = x >= 0 && x < a.V;
        if (yes) {
          const float p = a.target[(row0 + i) * a.target_stride + x];
          const float q = a.draft ? a.draft[(size_t)(d0 + i) * a.draft_stride + x] : 1.f;
          yes = (double)a.accept_u[d0 + i] * (double)q < (double)p;
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !yes);
      if (no) taken = i0 + __ffs(no) - 1;
    }
    if (lane == 0) s_taken = taken;
    if (rank == 0) {
      if (lane == 0) a.accepted[b] = taken;
      for (int i = lane; i <= n; i += 32) {
        const int x = i < n ? a.draft_tokens[d0 + i] : 0;
        if (x < 0 || x >= a.V) raise_status(a.dev_status, KDA_DEV_BAD_TOKEN);  // (behind a rejection too)
        if (i != taken) a.tokens[row0 + i] = i < taken ? x : -1;
      }
    }
  }
  __syncthreads();
  const int taken = s_taken;
  Weights w;
  w.p = a.target + (row0 + taken) * a.target_stride;
  w.q = taken < n && a.draft ? a.draft + (size_t)(d0 + taken) * a.draft_stride : nullptr;
  w.skip = taken < n && !a.draft ? a.draft_tokens[d0 + taken] : -1;

  // ---- the sum of this warp's segment
  const int seg = segment_of(a.V, segments);
  const int segment = rank * kWarps + warp;
  const int lo = (int)min((long long)a.V, (long long)segment * seg), hi = (int)min((long long)a.V, (long long)lo + seg);
  const int step = block_of(hi - lo);
  Sum mine = {};
#pragma unroll 1
  for (int i = 0; i < kBlocks; ++i) {
    const int from = min(hi, lo + i * step), to = min(hi, from + step);
    if constexpr (!kLong) {
      const Pair x = lane_sum<kVec>(w, from, to, lane);
      s_lane[i][tid] = x;
      add(mine, x.hi, x.lo);
    } else {
      double sum = 0.0;
      for (int at = from; at < to;) {
        Pair some = {0.f, 0.f};
#pragma unroll 1
        for (int run = 0; run < kRuns && at < to; ++run, at += 32 * kRun) {
          const Pair x = lane_sum<kVec>(w, at, min(to, at + 32 * kRun), lane);
          add(some, x.hi, x.lo);
        }
        sum += (double)some.hi + (double)some.lo;
      }
      s_lane[i][tid] = sum;
      mine += sum;
    }
  }
  const double sum = warp_total(mine);
  if (lane == 0) s_own[warp] = sum;
  cluster.sync();
  // ---- the segment that holds the drawn token: two per lane, scanned by every CTA's
  // first warp
  if (warp == 0) {
    const int i0 = 2 * lane, i1 = 2 * lane + 1;
    const double x0 = i0 < segments ? cluster.map_shared_rank(s_own, i0 / kWarps)[i0 % kWarps] : 0.0;
    const double x1 = i1 < segments ? cluster.map_shared_rank(s_own, i1 / kWarps)[i1 % kWarps] : 0.0;
    const double c1 = warp_scan(x0 + x1, lane), c0 = c1 - x1;
    const double all = __shfl_sync(0xffffffffu, c1, 31);
    const bool some = all > 0.0 && all <= 1e300;  // else nothing to draw from, or an infinity
    const double target = (double)a.sample_u[b] * all;
    const int l = first_past(c1, x0 + x1, target);
    if (lane == l) {
      const bool second = x1 > 0.0 && !(x0 > 0.0 && c0 > target);
      s_found = some ? 2 * l + (second ? 1 : 0) : -1;
      s_base = second ? c1 - x1 : c0 - x0;  // the running sum before the segment
      s_target = target;
    }
  }
  cluster.sync();  // (also: every s_own has been read, so a CTA may leave)
  if (s_found < 0 && rank == 0 && tid == 0) {
    a.tokens[row0 + taken] = -1;
    raise_status(a.dev_status, KDA_DEV_BAD_PROB);
  }
  if (s_found != segment) return;
  const double target = s_target;
  double base = s_base;

  // ---- within the segment (one warp per request): the block, the lane's run of
  // entries, the entry
  double part = 0.0;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const double x = warp_total(s_lane[i][tid]);
    if (lane == i) part = x;
  }
  double c = base + warp_scan(part, lane);
  int l = first_past(c, part, target);
  base = __shfl_sync(0xffffffffu, c - part, l);
  const int from = min(hi, lo + l * step), to = min(hi, from + step);
  const int each = (to - from + 31) / 32;
  const int v0 = min(to, from + lane * each), v1 = min(to, v0 + each);
  part = 0.0;
#pragma unroll 8
  for (int v = v0; v < v1; ++v) {
    float dh, dl;
    w.load(v, dh, dl);
    part += (double)dh + (double)dl;
  }
  c = base + warp_scan(part, lane);
  l = first_past(c, part, target);
  if (lane != l) return;
  c -= part;
  int drawn = -1;
  for (int v = v0; v < v1; ++v) {
    float dh, dl;
    w.load(v, dh, dl);
    const double x = (double)dh + (double)dl;
    if (!(x > 0.0)) continue;
    c += x;
    drawn = v;  // the last with a weight, should rounding let none pass
    if (c > target) break;
  }
  a.tokens[row0 + taken] = drawn;
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t stream) {
  int size = kMaxCluster;
  while (size > 1 && (long long)a.B * size > kSms * kCtasPerSm) size /= 2;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft)) & 15) == 0 &&
                   a.target_stride % 4 == 0 && (!a.draft || a.draft_stride % 4 == 0);
  const long long ctas = (long long)a.B * size;
  const bool runs = block_of(segment_of(a.V, kWarps * size)) > 32 * kRun;
  void (*kernel)(VerifyArgs, int) = runs ? (vec ? verify_kernel<true, true> : verify_kernel<false, true>)
                                         : (vec ? verify_kernel<true, false> : verify_kernel<false, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, size);
}

}  // namespace kda
