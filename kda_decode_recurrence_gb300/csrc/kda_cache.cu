// kda_cache.cu -- K and V rows into a paged cache (kda_cache_append) and back
// out of it (kda_cache_read).
//
//   append   s = amax_d |x_d| / 448 (1 for a row of zeros, NaN for a row with a
//            non-finite entry), code_d = e4m3(x_d / s), both divisions rounded
//            to nearest in fp32, the code to nearest even; or bf16 rows as they are
//   read     x_d = bf16(code_d * s)
//
// Both move about two bytes per operation, so HBM bounds them.  Lanes of 16 bytes (8 or 16
// to a row) take rows of consecutive tokens, the places of 32 of them looked up by a warp
// at once, four rows in flight per lane.  42156 tokens of prompts, 8 heads of 128,
// e4m3: 262 MB in 57 us, 4.6 TB/s (a copy: 6.7); the schedulers issue in 72% of their cycles
// (ALU 60%, DRAM 49%): three packed operations per quotient of two entries, and a row's place.
// In bf16: 345 MB in 56 us, 6.2 TB/s.  63691 rows back: 395 MB in 71 us, 5.6 TB/s; bf16 522 MB
// in 84 us, 6.2 TB/s.  64 single tokens: 10 us, the host's call.
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_paged.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.0f;

// Request of packed row t: the b with cu[b] <= t < cu[b + 1].  For a malformed
// cu the result is still in 0..B-1 and the caller's range check rejects it.
__device__ __forceinline__ int find_request(const int32_t* cu, int B, int t) {
  int lo = 0, hi = B - 1;  // the answer lies in lo..hi
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (fresh(cu + mid + 1) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Whether request b with rows t0 .. t1 - 1 and at[b] = `at` is well formed.
template <bool kAppend>
__device__ __forceinline__ bool good_request(const CacheRowsArgs& p, int t0, int t1, long long at) {
  return t0 >= 0 && t1 >= t0 && t1 <= p.T && at >= 0 &&
         (kAppend ? at : at + (t1 - t0)) <= (long long)p.c.max_pages * p.c.page_size;
}

// By one more CTA, beside those that take rows: every request that is not well formed is
// reported, whether or not a row shows it, and so are offsets that do not span the T rows.
template <bool kAppend>
__device__ __forceinline__ void check_requests(const CacheRowsArgs& p) {
  bool bad = threadIdx.x == 0 && (fresh(p.cu) != 0 || fresh(p.cu + p.B) != p.T);
  for (unsigned b = threadIdx.x; b < (unsigned)p.B; b += kThreads)
    bad |= !good_request<kAppend>(p, fresh(p.cu + b), fresh(p.cu + b + 1), p.at ? fresh(p.at + b) : 0);
  if (bad) raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
}

// Page and offset of packed row t; page -1: the row has no place.
template <bool kAppend>
__device__ __forceinline__ int2 find_place(const CacheRowsArgs& p, int t) {
  const int2 none = make_int2(-1, 0);
  const int b = find_request(p.cu, p.B, t);
  const int t0 = fresh(p.cu + b), t1 = fresh(p.cu + b + 1);
  const long long at = p.at ? fresh(p.at + b) : 0;
  if (t < t0 || t >= t1 || !good_request<kAppend>(p, t0, t1, at)) return none;
  const long long pos = kAppend ? at - (t1 - t) : at + (t - t0);
  if (pos < 0) return none;  // padding before the sequence's first position
  const int page = fresh(p.c.page_table + (size_t)b * p.c.max_pages + pos / p.c.page_size);
  if (page < 0 || page >= p.c.num_pages) {
    raise_status(p.dev_status, KDA_DEV_BAD_PAGE);
    return none;
  }
  return make_int2(page, (int)(pos % p.c.page_size));
}

// A warp takes `tokens` consecutive tokens: each lane looks up the place of one, then
// all their rows follow, kLanes lanes (8 entries each) to a row and kUnroll rows per
// lane in flight.
struct Split {
  int tokens;      // per warp, at most 32
  uint32_t inv;    // ceil(2^32 / (2 HKV)): r / (2 HKV) = umulhi(r, inv) for the warp's rows r
};
constexpr int kUnroll = 4;

template <int D>
struct Rows {
  static constexpr int kLanes = D / 8;
  static constexpr int kPerWarp = 32 / kLanes;

  int t0, rows, sub, mine;
  int2 place;  // this lane's token's

  template <bool kAppend>
  __device__ __forceinline__ bool start(const CacheRowsArgs& p, const Split& s) {
    const int lane = threadIdx.x & 31;
    const long long first = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * s.tokens;
    if (first >= p.T) return false;
    t0 = (int)first;
    const int tokens = min(s.tokens, p.T - t0);
    rows = tokens * 2 * p.c.HKV;
    sub = lane % kLanes;
    mine = lane / kLanes;
    place = lane < tokens ? find_place<kAppend>(p, t0 + lane) : make_int2(-1, 0);
    return true;
  }
  struct Row {
    int t, h, page;    // token, key head, page (-1: none)
    bool is_v;
    size_t at;         // row of the cache
  };
  __device__ __forceinline__ Row row(const CacheRowsArgs& p, const Split& s, int r) const {
    Row x;
    const int i = min((int)__umulhi((uint32_t)r, s.inv), 31);
    const int in = r - i * 2 * p.c.HKV;
    x.is_v = in >= p.c.HKV;
    x.h = x.is_v ? in - p.c.HKV : in;
    x.t = t0 + i;
    x.page = __shfl_sync(0xffffffffu, place.x, i);
    const int off = __shfl_sync(0xffffffffu, place.y, i);
    x.at = ((size_t)max(x.page, 0) * p.c.HKV + x.h) * p.c.page_size + off;
    return x;
  }
};

// 1 / s within two roundings, for s far from the ends of fp32's range.
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(fmaf(-s, r, 1.f), r, r);
}
// x / s rounded to nearest, nr = -1 / s: one correction by the exact remainder
// (Markstein), the remainder with the sign that lets a zero keep its own.
__device__ __forceinline__ float quotient(float x, float s, float nr) {
  const float y = x * -nr;
  return fmaf(fmaf(s, y, -x), nr, y);
}
__device__ __forceinline__ float2 quotient2(float2 x, float2 s, float2 r, float2 nr) {
  const float2 y = __fmul2_rn(x, r);
  return __ffma2_rn(__ffma2_rn(s, y, make_float2(-x.x, -x.y)), nr, y);
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 4) cache_append_kernel(const CacheRowsArgs p, const Split split) {
  using R = Rows<D>;
  R rows;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) return check_requests<true>(p);
  if (!rows.template start<true>(p, split)) return;
  for (int base = 0; base < rows.rows; base += R::kPerWarp * kUnroll) {
    uint4 x[kUnroll];
    typename R::Row row[kUnroll];
    bool live[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = base + u * R::kPerWarp + rows.mine;
      live[u] = r < rows.rows;
      row[u] = rows.row(p, split, live[u] ? r : 0);
      const kda_bf16* src = row[u].is_v ? p.v_rows + row[u].t * p.v_stride : p.k_rows + row[u].t * p.k_stride;
      x[u] = fresh(reinterpret_cast<const uint4*>(src + (size_t)row[u].h * D + rows.sub * 8));
      live[u] = live[u] && row[u].page >= 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      void* cache = row[u].is_v ? p.c.v : p.c.k;
      if constexpr (!kE4m3) {
        if (live[u]) *reinterpret_cast<uint4*>(static_cast<kda_bf16*>(cache) + row[u].at * D + rows.sub * 8) = x[u];
      } else {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
#pragma unroll
        for (int o = R::kLanes / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = max(top & 0xffffu, top >> 16);
        const bool finite = top < 0x7f80u;
        // (the largest entry from 2^-50 to 2^69: everything in fp32's normal range)
        const bool usual = top - 0x2680u < 0x6200u - 0x2680u;
        float s, y[8];
        if (usual) {
          s = quotient(__uint_as_float(top << 16), kE4m3Max, -1.f / kE4m3Max);
          const float r = reciprocal(s);
          const float2 s2 = make_float2(s, s), r2 = make_float2(r, r), nr2 = make_float2(-r, -r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 z = quotient2(make_float2(bf16_lo(w[i]), bf16_hi(w[i])), s2, r2, nr2);
            y[2 * i] = z.x;
            y[2 * i + 1] = z.y;
          }
        } else {
          s = !finite ? __uint_as_float(0x7fffffffu) : top == 0 ? 1.0f : __fdiv_rn(__uint_as_float(top << 16), kE4m3Max);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // (zeros where the scale says it all: a code that is no number would reach tokens
            // that do not see the row, 0 x NaN)
            y[2 * i] = finite ? __fdiv_rn(bf16_lo(w[i]), s) : 0.f;
            y[2 * i + 1] = finite ? __fdiv_rn(bf16_hi(w[i]), s) : 0.f;
          }
        }
        uint32_t code[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          code[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_SATFINITE,
                                                             __NV_E4M3) << (16 * (i & 1));
        if (live[u]) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row[u].at * D + rows.sub * 8) =
              make_uint2(code[0], code[1]);
          if (rows.sub == 0) (row[u].is_v ? p.c.v_scale : p.c.k_scale)[row[u].at] = s;
        }
      }
    }
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 6) cache_read_kernel(const CacheRowsArgs p, const Split split) {
  using R = Rows<D>;
  R rows;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) return check_requests<false>(p);
  if (!rows.template start<false>(p, split)) return;
  for (int base = 0; base < rows.rows; base += R::kPerWarp * kUnroll) {
    uint4 x[kUnroll];
    float s[kUnroll];
    typename R::Row row[kUnroll];
    bool live[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = base + u * R::kPerWarp + rows.mine;
      live[u] = r < rows.rows;
      row[u] = rows.row(p, split, live[u] ? r : 0);
      x[u] = make_uint4(0, 0, 0, 0);
      s[u] = 0.f;
      const void* cache = row[u].is_v ? p.c.v : p.c.k;
      if (live[u] && row[u].page >= 0) {
        if constexpr (kE4m3) {
          const uint2 c = fresh(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) +
                                                               row[u].at * D + rows.sub * 8));
          x[u].x = c.x;
          x[u].y = c.y;
          s[u] = fresh((row[u].is_v ? p.c.v_scale : p.c.k_scale) + row[u].at);
        } else {
          x[u] = fresh(reinterpret_cast<const uint4*>(static_cast<const kda_bf16*>(cache) +
                                                      row[u].at * D + rows.sub * 8));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if constexpr (kE4m3) {
        const uint32_t c[2] = {x[u].x, x[u].y};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t pair = (c[i >> 1] >> (16 * (i & 1))) & 0xffffu;
          const __half2 y(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3));
          const float2 f = __half22float2(y);
          const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s[u], f.y * s[u]);
          o[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        x[u] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      kda_bf16* out = row[u].is_v ? p.v_rows + row[u].t * p.v_stride : p.k_rows + row[u].t * p.k_stride;
      if (live[u]) *reinterpret_cast<uint4*>(out + (size_t)row[u].h * D + rows.sub * 8) = x[u];
    }
  }
}

// As many tokens to a warp as leave every SM 128 of them (one look-up then serves
// several rows in flight; fewer warps leave a tail), eight at most.
template <typename Kernel>
cudaError_t run(Kernel kernel, const CacheRowsArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  constexpr int kAllWarps = 152 * 128;
  Split s;
  s.tokens = a.T / kAllWarps < 1 ? 1 : a.T / kAllWarps > 8 ? 8 : a.T / kAllWarps;
  s.inv = (uint32_t)(((1ull << 32) + 2 * a.c.HKV - 1) / (2 * a.c.HKV));
  const long long per_cta = (long long)(kThreads / 32) * s.tokens;
  // (the last CTA looks at the requests)
  return launch(kernel, dim3((unsigned)((a.T + per_cta - 1) / per_cta) + 1), dim3(kThreads), 0, stream, true, a, s);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsArgs& a, cudaStream_t stream) {
  if (a.c.D == 128)
    return a.c.e4m3 ? run(cache_append_kernel<128, true>, a, stream)
                    : run(cache_append_kernel<128, false>, a, stream);
  return a.c.e4m3 ? run(cache_append_kernel<64, true>, a, stream)
                  : run(cache_append_kernel<64, false>, a, stream);
}

cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t stream) {
  if (a.c.D == 128)
    return a.c.e4m3 ? run(cache_read_kernel<128, true>, a, stream)
                    : run(cache_read_kernel<128, false>, a, stream);
  return a.c.e4m3 ? run(cache_read_kernel<64, true>, a, stream)
                  : run(cache_read_kernel<64, false>, a, stream);
}

}  // namespace kda
