// Pieces shared by the attention kernels over the paged 8-bit cache.
#pragma once

#include <float.h>

#include "kv_common.cuh"

namespace moe {

// Rows (new tokens of a sequence x query heads of a kv head) up to which a
// sequence is split over its keys by kv_decode_kernel; with more, its rows fill
// the 128-row tiles of kv_prefill_kernel.
constexpr int kDecodeRows = 32;
constexpr int kDecodeCounters = 3 * 1024;   // int32, at the start of the workspace

struct AttnArgs {
  moe_kv_attention_desc d;
  int32_t G;          // query heads per kv head
  float* parts;       // partial results of split rows
  int32_t* counters;  // arrivals at a split's parts, zero between calls
};

int kv_decode_launch(const AttnArgs& a, int64_t max_rows, cudaStream_t st);
// Bytes of parts that each may leave (one after the other, in the same place).
size_t kv_decode_workspace();
size_t kv_prefill_workspace();
int kv_prefill_launch(const AttnArgs& a, cudaStream_t st);

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Weights are exponentials relative to a reference kHead powers of two below the running
// maximum, which follows it only once a weight would reach 2^kLazy: weights stay inside
// f16, and what a row has so far is rescaled rarely.  f16 is normal down to 2^-14, so a
// weight keeps its 11 bits down to 2^-22 of the row's largest, and below that is rounded
// to multiples of 2^-32 of it, so that keys by the thousand under a dominant one still
// count.  (With the reference at the maximum those were 2^-14 and 2^-24.)
constexpr float kHead = 8.0f, kLazy = 15.5f;
// A V scale this small counts as this: weights carry the scale as its logarithm, and the
// sum of weights over scales, up to 2^kLazy times 2^31 keys over this, has to stay in fp32.
constexpr float kMinScale = 8.2718061e-25f;   // 2^-80

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// V scales ride in the weights, which are f16, so where they lie far apart a page with
// small values has to be kept from falling under a large one's: outputs may be its alone.
// Scales within 2^kNear of each other count as one size.
constexpr int kNear = 4;

// cap * log2(e) * tanh(y) for y = score / cap: tanh(y) = 1 - 2 / (exp(2y) + 1),
// which ends at +-1 for any y and passes NaN on.  Its error is absolute, some 2^-22 of
// the cap, however small the score: for caps up to kCapDirect, where that is below 2^-15.
__device__ __forceinline__ float capped_log2(float y, float cap_log2) {
  const float e = ex2(2.0f * kLog2e * y);
  return fmaf(-2.0f * cap_log2, __fdividef(1.0f, e + 1.0f), cap_log2);
}
// Larger caps take tanh(y) / y times the score, whose error is relative to the score:
// below |y| = 1/4 by the series 1 - y^2/3 + 2 y^4/15 - 17 y^6/315 + 62 y^8/2835, whose
// next term is below 2^-26 there.
constexpr float kCapDirect = 64.0f;
__device__ __forceinline__ float tanh_ratio(float y) {
  const float z = y * y;
  const float p = fmaf(fmaf(fmaf(z, 62.0f / 2835.0f, -17.0f / 315.0f), z, 2.0f / 15.0f), z, -1.0f / 3.0f);
  const float large = fmaf(-2.0f, __fdividef(1.0f, ex2(2.0f * kLog2e * y) + 1.0f), 1.0f);
  return fabsf(y) < 0.25f ? fmaf(z, p, 1.0f) : __fdividef(large, y);
}
// Caps beyond these are as good as these: below, no score differs from 0 in a weight;
// above, none is bent within fp32 that is below 2^50.  In between score / cap and its
// factors stay in fp32's range.
constexpr float kMinCap = 9.3132257e-10f, kMaxCap = 1.8446744e19f;   // 2^-30, 2^64

// What a sequence's part of the descriptors says, checked.
struct Seq {
  int n, len, c0;   // n = 0: no rows to compute
};

__device__ __forceinline__ Seq load_seq(const moe_kv_attention_desc& d, int b, int32_t* bad) {
  Seq s;
  s.c0 = __ldg(d.cache.cu_new + b);
  const int c1 = __ldg(d.cache.cu_new + b + 1);
  s.len = __ldg(d.cache.kv_len + b);
  s.n = c1 - s.c0;
  if (s.n == 0) return s;
  if (s.c0 < 0 || s.n < 0 || c1 > d.T || s.len < s.n) {
    *bad |= MOE_DEV_BAD_INDEX;
    s.n = 0;
  } else if ((s.len - 1) / d.cache.page_size >= d.cache.max_pages || (d.max_q && s.n > d.max_q)) {
    *bad |= MOE_DEV_OVERFLOW;
    s.n = 0;
  }
  return s;
}

// First key that new token i of a sequence sees, and one past the last.
__device__ __forceinline__ int first_key(const moe_kv_attention_desc& d, const Seq& s, int i) {
  return d.window > 0 ? max(0, s.len - s.n + i - d.window + 1) : 0;
}
__device__ __forceinline__ int end_key(const moe_kv_attention_desc& d, const Seq& s, int i) {
  return (d.flags & MOE_KV_FULL) ? s.len : s.len - s.n + i + 1;
}

// Power of two that takes a row's largest |element| into [1, 2), and its
// inverse; a row with a non-finite element gets a NaN inverse, so that its
// scores, and its output, are NaN.
__device__ __forceinline__ void row_scale(float amax, float& mul, float& inv) {
  const uint32_t e = __float_as_uint(amax) >> 23;           // amax >= 0
  if (e == 255) {
    mul = 0.0f;
    inv = __uint_as_float(0x7FC00000u);
  } else {
    const uint32_t c = min(max(e, 4u), 250u);               // both factors stay normal numbers
    mul = __uint_as_float((254u - c) << 23);
    inv = __uint_as_float(c << 23);
  }
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 0x80 in each byte of w that holds a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

}  // namespace
}  // namespace moe
