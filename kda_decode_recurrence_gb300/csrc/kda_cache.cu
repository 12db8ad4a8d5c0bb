// kda_cache.cu -- K and V rows into a paged cache (kda_cache_append) and back
// out of it (kda_cache_read).
//
//   append   s = amax_d |x_d| / 448 (1 for a row of zeros, NaN for a row with a
//            non-finite entry), code_d = e4m3(x_d / s), both divisions rounded
//            to nearest in fp32, the code to nearest even; or bf16 rows as they are
//   read     x_d = bf16(code_d * s)
//
// Both move about two bytes per operation, so HBM bounds them.
#include <cuda_fp8.h>

#include "kda_common.cuh"
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
    if (__ldg(cu + mid + 1) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Page and offset of packed row t; page -1: the row has no place.
template <bool kAppend>
__device__ __forceinline__ int2 find_place(const CacheRowsArgs& p, int t) {
  const int2 none = make_int2(-1, 0);
  const int b = find_request(p.cu, p.B, t);
  const int t0 = __ldg(p.cu + b), t1 = __ldg(p.cu + b + 1);
  if (t < t0 || t >= t1 || t0 < 0 || t1 > p.T) {
    raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
    return none;
  }
  const long long at = p.at ? __ldg(p.at + b) : 0;
  const long long capacity = (long long)p.c.max_pages * p.c.page_size;
  if (at < 0 || (kAppend ? at : at + (t1 - t0)) > capacity) {
    raise_status(p.dev_status, KDA_DEV_BAD_SEQLEN);
    return none;
  }
  const long long pos = kAppend ? at - (t1 - t) : at + (t - t0);
  if (pos < 0) return none;  // padding before the sequence's first position
  const int page = __ldg(p.c.page_table + (size_t)b * p.c.max_pages + pos / p.c.page_size);
  if (page < 0 || page >= p.c.num_pages) {
    raise_status(p.dev_status, KDA_DEV_BAD_PAGE);
    return none;
  }
  return make_int2(page, (int)(pos % p.c.page_size));
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const CacheRowsArgs p) {
  constexpr int kLanes = D / 8;  // lanes per row, 8 elements each
  constexpr int kRows = kThreads / kLanes;
  const int sub = threadIdx.x % kLanes;
  const long long rows = 2ll * p.T * p.c.HKV;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kLanes;
  const bool live = row < rows;
  const long long r = live ? row : 0;
  const int h = (int)(r % p.c.HKV);
  const bool is_v = (r / p.c.HKV) & 1;
  const int t = (int)(r / (2 * p.c.HKV));
  const int2 place = find_place<true>(p, t);
  const kda_bf16* src = is_v ? p.v_rows + t * p.v_stride : p.k_rows + t * p.k_stride;
  const uint4 x = *reinterpret_cast<const uint4*>(src + (size_t)h * D + sub * 8);
  const size_t dst = ((size_t)max(place.x, 0) * p.c.HKV + h) * p.c.page_size + place.y;
  void* cache = is_v ? p.c.v : p.c.k;
  if (!kE4m3) {
    if (live && place.x >= 0)
      *reinterpret_cast<uint4*>(static_cast<kda_bf16*>(cache) + dst * D + sub * 8) = x;
    return;
  }
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool finite = top < 0x7f80u;
  const float s = !finite ? __uint_as_float(0x7fffffffu)
                  : top == 0 ? 1.0f : __fdiv_rn(__uint_as_float(top << 16), kE4m3Max);
  uint32_t code[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = make_float2(__fdiv_rn(bf16_lo(w[i]), s), __fdiv_rn(bf16_hi(w[i]), s));
    code[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
  }
  if (live && place.x >= 0) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + dst * D + sub * 8) =
        make_uint2(code[0], code[1]);
    if (sub == 0) (is_v ? p.c.v_scale : p.c.k_scale)[dst] = s;
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheRowsArgs p) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = kThreads / kLanes;
  const int sub = threadIdx.x % kLanes;
  const long long rows = 2ll * p.T * p.c.HKV;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kLanes;
  if (row >= rows) return;
  const int h = (int)(row % p.c.HKV);
  const bool is_v = (row / p.c.HKV) & 1;
  const int t = (int)(row / (2 * p.c.HKV));
  const int2 place = find_place<false>(p, t);
  uint4 x = make_uint4(0, 0, 0, 0);
  if (place.x >= 0) {
    const size_t src = ((size_t)place.x * p.c.HKV + h) * p.c.page_size + place.y;
    const void* cache = is_v ? p.c.v : p.c.k;
    if (kE4m3) {
      const uint2 code = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + src * D + sub * 8);
      const float s = (is_v ? p.c.v_scale : p.c.k_scale)[src];
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t pair = ((i < 2 ? code.x : code.y) >> (16 * (i & 1))) & 0xffffu;
        const __half2 y(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3));
        const float2 f = __half22float2(y);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      x = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      x = *reinterpret_cast<const uint4*>(static_cast<const kda_bf16*>(cache) + src * D + sub * 8);
    }
  }
  kda_bf16* out = is_v ? p.v_rows + t * p.v_stride : p.k_rows + t * p.k_stride;
  *reinterpret_cast<uint4*>(out + (size_t)h * D + sub * 8) = x;
}

template <typename Kernel>
cudaError_t run(Kernel kernel, const CacheRowsArgs& a, cudaStream_t stream) {
  const long long rows = 2ll * a.T * a.c.HKV;
  const int per_cta = kThreads / (a.c.D / 8);
  const long long grid = (rows + per_cta - 1) / per_cta;
  if (grid == 0) return cudaSuccess;
  kernel<<<(unsigned)grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
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
