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
// sums are pairs of fp32 (hi + lo, about 48 bits) per lane and fp64 only where
// lanes are joined: the drawn token has to be the same for any order of
// summation, and neighbours in a large vocabulary lie 1e-6 of the sum apart.
#include <cooperative_groups.h>

#include "kda_common.cuh"
#include "kda_paged.h"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;                  // CTAs per request
constexpr int kSegments = kWarps * kCluster;  // a row is cut into one segment per warp
constexpr int kBlocks = 8;                   // blocks a segment is searched by

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

__device__ __forceinline__ double warp_total(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
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

// This lane's share of the weights lo..hi-1 (entries lo + lane, + 32, ...).
template <bool kHasQ>
__device__ __forceinline__ Pair lane_sum(const Weights& w, int lo, int hi, int lane) {
  constexpr int kUnroll = 8;
  Pair s = {0.f, 0.f};
  int v = lo + lane;
  for (; v + 32 * (kUnroll - 1) < hi; v += 32 * kUnroll) {
    float pv[kUnroll], qv[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) pv[i] = __ldg(w.p + v + 32 * i);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) qv[i] = kHasQ ? __ldg(w.q + v + 32 * i) : 0.f;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      float d, e;
      w.get(pv[i], qv[i], v + 32 * i, d, e);
      add(s, d, e);
    }
  }
  for (; v < hi; v += 32) {
    float d, e;
    w.get(__ldg(w.p + v), kHasQ ? __ldg(w.q + v) : 0.f, v, d, e);
    add(s, d, e);
  }
  return s;
}

__device__ __forceinline__ double total(const Pair& s) { return (double)s.hi + (double)s.lo; }

// The first lane with a weight x whose inclusive running sum c passes `target`;
// if rounding lets none pass, the last lane with a weight (0: no weight at all).
__device__ __forceinline__ int first_past(double c, double x, double target) {
  const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
  const unsigned past = __ballot_sync(0xffffffffu, c > target) & some;
  return past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    verify_kernel(const VerifyArgs a) {
  __shared__ int s_taken;
  __shared__ double s_own[kWarps];
  __shared__ double s_all[kSegments];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int b = blockIdx.x / kCluster;
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
        } else if (rank == 0) {
          raise_status(a.dev_status, KDA_DEV_BAD_TOKEN);
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !yes);
      if (no) taken = i0 + __ffs(no) - 1;
    }
    if (lane == 0) s_taken = taken;
    if (rank == 0) {
      if (lane == 0) a.accepted[b] = taken;
      for (int i = lane; i <= n; i += 32)
        if (i != taken) a.tokens[row0 + i] = i < taken ? a.draft_tokens[d0 + i] : -1;
    }
  }
  __syncthreads();
  const int taken = s_taken;
  Weights w;
  w.p = a.target + (row0 + taken) * a.target_stride;
  w.q = taken < n && a.draft ? a.draft + (size_t)(d0 + taken) * a.draft_stride : nullptr;
  w.skip = taken < n && !a.draft ? a.draft_tokens[d0 + taken] : -1;

  // ---- the sum of this warp's segment
  const int seg = (a.V + kSegments - 1) / kSegments;
  const int segment = rank * kWarps + warp;
  const int lo = min((long long)a.V, (long long)segment * seg), hi = min(a.V, lo + seg);
  const Pair mine = w.q ? lane_sum<true>(w, lo, hi, lane) : lane_sum<false>(w, lo, hi, lane);
  const double sum = warp_total(total(mine));
  if (lane == 0) s_own[warp] = sum;
  cluster.sync();
  if (tid < kSegments) s_all[tid] = cluster.map_shared_rank(s_own, tid / kWarps)[tid % kWarps];
  cluster.sync();  // (also: every s_own has been read, so a CTA may leave)

  // ---- the segment that holds the drawn token: two per lane, scanned
  const double x0 = s_all[2 * lane], x1 = s_all[2 * lane + 1];
  const double c1 = warp_scan(x0 + x1, lane), c0 = c1 - x1;
  const double all = __shfl_sync(0xffffffffu, c1, 31);
  if (!(all > 0.0) || all > 1e300) {  // nothing to draw from, or an infinity
    if (rank == 0 && tid == 0) {
      a.tokens[row0 + taken] = -1;
      raise_status(a.dev_status, KDA_DEV_BAD_PROB);
    }
    return;
  }
  const double target = (double)a.sample_u[b] * all;
  int l = first_past(c1, x0 + x1, target);
  // the two halves of that lane
  const double b1 = __shfl_sync(0xffffffffu, c1, l), b0 = __shfl_sync(0xffffffffu, c0, l);
  const double h0 = __shfl_sync(0xffffffffu, x0, l), h1 = __shfl_sync(0xffffffffu, x1, l);
  const bool second = h1 > 0.0 && !(h0 > 0.0 && b0 > target);
  const int found = 2 * l + (second ? 1 : 0);
  if (found != segment) return;
  double base = second ? b1 - h1 : b0 - h0;  // the running sum before the segment

  // ---- within the segment (one warp per request): the block, then the entry
  const int step = (((hi - lo) + kBlocks - 1) / kBlocks + 31) & ~31;
  double part = 0.0;
  for (int i = 0; i < kBlocks; ++i) {
    const int from = min(hi, lo + i * step), to = min(hi, from + step);
    const double x = warp_total(total(w.q ? lane_sum<true>(w, from, to, lane) : lane_sum<false>(w, from, to, lane)));
    if (lane == i) part = x;
  }
  double c = base + warp_scan(part, lane);
  l = first_past(c, part, target);
  base = __shfl_sync(0xffffffffu, c - part, l);
  const int from = lo + l * step, to = min(hi, from + step);
  int drawn = -1;
  for (int v0 = from; v0 < to; v0 += 32) {
    float dh = 0.f, dl = 0.f;
    if (v0 + lane < to) w.load(v0 + lane, dh, dl);
    const double x = (double)dh + (double)dl;
    c = base + warp_scan(x, lane);
    const unsigned past = __ballot_sync(0xffffffffu, c > target);
    const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
    if (past & some) {
      drawn = v0 + __ffs(past & some) - 1;
      break;
    }
    if (some) drawn = v0 + 31 - __clz(some);  // the last with a weight so far
    base = __shfl_sync(0xffffffffu, c, 31);
  }
  if (lane == 0) a.tokens[row0 + taken] = drawn;
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t stream) {
  verify_kernel<<<(unsigned)a.B * kCluster, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
