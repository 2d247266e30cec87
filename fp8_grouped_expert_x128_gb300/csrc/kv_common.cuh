// Pieces shared by the key/value cache kernels: descriptor checks, the search
// for a row's sequence, and conversions of the element types.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {
namespace {

inline bool kv_strides_ok(int64_t a, int64_t b, int64_t c, int64_t unit) {
  return a >= 0 && b >= 0 && c >= 0 && a % unit == 0 && b % unit == 0 && c % unit == 0;
}

inline int check_kv_cache(const moe_kv_cache& c, int64_t T) {
  MOE_CHECK_ARG(c.batch >= 0 && c.pages >= 0 && c.max_pages >= 0 && c.kv_heads >= 1 && T >= 0);
  MOE_CHECK_ARG(c.dtype == MOE_DTYPE_BF16 || c.dtype == MOE_DTYPE_F16);
  MOE_CHECK_ARG(kv_strides_ok(c.k_page_ld, c.k_head_ld, c.k_slot_ld, 16));
  MOE_CHECK_ARG(kv_strides_ok(c.v_page_ld, c.v_head_ld, c.v_slot_ld, 16));
  MOE_CHECK_ARG(c.table_ld >= 0);
  if (c.dim != 64 && c.dim != 128) return MOE_ERR_UNSUPPORTED;
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128) return MOE_ERR_UNSUPPORTED;
  // positions, rows and units of work are 32-bit numbers; the kernels look up pages some
  // thousand positions ahead of a sequence's end, which must not wrap around
  constexpr int32_t kMaxTokens = INT32_MAX - 65535;
  if (c.batch > (1 << 20) || T > (1 << 24) || c.kv_heads > 1024 || c.pages > INT32_MAX ||
      c.max_pages > kMaxTokens / c.page_size || c.k_page_ld >= (1ll << 35) || c.v_page_ld >= (1ll << 35))
    return MOE_ERR_UNSUPPORTED;
  if (T == 0 || c.batch == 0) return MOE_OK;
  MOE_CHECK_ARG(c.k && c.v && c.k_scale && c.v_scale && c.page_table && c.cu_new && c.kv_len);
  MOE_CHECK_ARG(aligned16(c.k) && aligned16(c.v));
  return MOE_OK;
}

// Largest b in [0, n) with f(b) <= x, for f not decreasing and f(0) <= x (else
// 0): 32 probes a round by the lanes of a warp, every lane gets the answer.
template <class F>
__device__ __forceinline__ int warp_find(int n, int x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lo + lane * step;
    const bool le = lane * step < len && f(at) <= x;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;
    len = min(step, len - k * step);
    lo += k * step;
  }
  return lo;
}

template <bool F16>
__device__ __forceinline__ float2 pair_to_float(uint32_t w) {
  if constexpr (F16) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t pair_from_float(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = pair_to_float<F16>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pair_from_float<F16>(f[0], f[1]), pair_from_float<F16>(f[2], f[3]),
                    pair_from_float<F16>(f[4], f[5]), pair_from_float<F16>(f[6], f[7]));
}

// Two E4M3 codes (the low one first) as two f16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}

}  // namespace
}  // namespace moe
