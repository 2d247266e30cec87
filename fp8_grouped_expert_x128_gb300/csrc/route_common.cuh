// Pieces of the routing kernels (moe_route): sortable keys, how near two values may
// lie, and the forms in 64 bits that decide where fp32 does not.
#pragma once

#include <cfloat>
#include <cmath>

#include "kv_common.cuh"

namespace moe {

// The kernel for many tokens, and which calls are for it.
bool is_for_route_many(const moe_route_desc& d);
int route_many(const moe_route_desc& d, int group_lanes, cudaStream_t st);

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// A logit as fp32: NaN and -inf (an expert that is not open) become -inf, +inf the
// largest fp32.
__device__ __forceinline__ float as_logit(float z) { return z > -INFINITY ? fminf(z, FLT_MAX) : -INFINITY; }

template <int DT>
__device__ __forceinline__ float raw_logit(const void* row, int e) {
  if constexpr (DT == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(row) + e);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(row) + e);
  return DT == MOE_DTYPE_F16 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b);
}
template <int DT>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  return as_logit(raw_logit<DT>(row, e));
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Numbers whose order as unsigned integers is that of the doubles (and -0 as 0); 0 is none.
// GB300 has few 64-bit floating-point units: values are compared as integers.
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double value_of(uint64_t k) {
  return __longlong_as_double(static_cast<int64_t>(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

// One token in 64-bit arithmetic by one warp.  value: E words of shared memory.
// Lane j < k gets the number of the j-th expert, -1 where there is none.
template <int DT>
__device__ __noinline__ int route_exact(const moe_route_desc& d, const void* row, uint64_t* value, int group_lanes) {
  const int lane = threadIdx.x & 31;
  const bool softmax = d.flags & MOE_ROUTE_SOFTMAX, pair = d.flags & MOE_ROUTE_GROUP_PAIR;
  float top = -INFINITY;
  double sum = 1.0;
  if (softmax) {
    for (int e = lane; e < d.E; e += 32) top = fmaxf(top, load_logit<DT>(row, e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    sum = 0.0;
    for (int e = lane; e < d.E; e += 32) {
      const float z = load_logit<DT>(row, e);
      if (z > -INFINITY) sum += exp(static_cast<double>(z) - top);
    }
    sum = warp_sum(sum);
  }
  auto score = [&](double z) { return softmax ? exp(z - top) / sum : 1.0 / (1.0 + exp(-z)); };
  auto fill = [&](bool scores) {
    for (int e = lane; e < d.E; e += 32) {
      const float z = load_logit<DT>(row, e);
      const float b = d.bias ? __ldg(d.bias + e) : 0.0f;
      uint64_t k = 0;
      if (z > -INFINITY && b > -INFINITY) k = key_of(scores ? score(z) + b : static_cast<double>(z));
      value[e] = k;
    }
    __syncwarp();
  };
  const int size = d.E / d.n_group;
  uint32_t kept = kAll;
  if (d.n_group > 1) {
    fill(d.bias != nullptr || pair);
    const int g = lane / group_lanes;
    uint64_t a = 0, b = 0;
    if (g < d.n_group)
      for (int i = lane % group_lanes; i < size; i += group_lanes) {
        const uint64_t v = value[g * size + i];
        b = max(b, min(a, v));
        a = max(a, v);
      }
    for (int o = group_lanes / 2; o > 0; o >>= 1) {
      const uint64_t oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    }
    if (pair && b != 0) a = key_of(value_of(a) + value_of(b));
    int rank = 0;
    for (int i = 0; i < d.n_group; ++i) {
      const uint64_t other = __shfl_sync(kAll, a, i * group_lanes);
      rank += other > a || (other == a && i < g);
    }
    kept = __ballot_sync(kAll, g < d.n_group && rank < d.topk_group);
    __syncwarp();
  }
  if (d.n_group == 1 || (d.bias == nullptr && pair)) fill(d.bias != nullptr);
  int found = -1;
  for (int j = 0; j < d.k; ++j) {
    uint64_t v = 0;
    int n = INT32_MAX;
    for (int e = lane; e < d.E; e += 32) {
      const uint64_t x = value[e];
      if (x > v && (d.n_group == 1 || ((kept >> (e / size * group_lanes)) & 1))) {
        v = x;
        n = e;
      }
    }
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    const uint64_t best = static_cast<uint64_t>(hi) << 32 | lo;
    if (best == 0) break;
    n = __reduce_min_sync(kAll, v == best ? n : INT32_MAX);
    if (lane == j) found = n;
    if (lane == (n & 31)) value[n] = 0;
    __syncwarp();
  }
  __syncwarp();
  return found;
}

// Numbers whose order as unsigned integers is that of the floats (and -0 as 0); 0 is none.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
// of a sum, which is never -0
__device__ __forceinline__ uint32_t key_of_sum(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Values this near may be in another order than they appear in.  A sigmoid: its exponential
// is off by at most 2^-22 + |z| 2^-24 relatively, its slope is at most 1/4 and |z| times its slope 0.23, its
// quotient is off by 2^-23: less than 2^-22 in all, 2^-21 between two of them.  A softmax's share:
// its sum is off by less than 2^-18.5 of it (32 additions one after another and 5 more), by which the
// difference of two shares shifts, at most the largest share; the exponentials, as shares of it, by
// less than 2^-21.  Adding a bias rounds either to 2^-24.
__device__ __forceinline__ float unit_of(bool softmax, float largest_share) { return softmax ? 0x1p-18f * largest_share : 0x1p-20f; }
__device__ __forceinline__ float near_of(float v, float unit) { return unit + 0x1p-22f * fabsf(v); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504088896340736f;

// A sigmoid below 2^-30 is its exponential in fp32: such a score, as a part of that of the largest of them.
// Past exp(709.78), which is past 64 bits, it is 0.
__device__ __forceinline__ float small_score(float x, float largest) { return x >= -709.78f ? expf(x - largest) : 0.0f; }

// A logit's score in 64 bits, for a warp that has the token's row.  What a softmax needs is looked
// for here and not handed over: few tokens come here, and all would keep it in registers.
template <int DT, bool kSoftmax>
struct ExactScore {
  float top = -INFINITY;
  double sum = 0.0;
  __device__ __forceinline__ ExactScore(const void* row, int E) {
    if constexpr (kSoftmax) {
      const int lane = threadIdx.x & 31;
      for (int e = lane; e < E; e += 32) top = fmaxf(top, load_logit<DT>(row, e));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
#pragma unroll 4
      for (int e = lane; e < E; e += 32) {
        const float z = load_logit<DT>(row, e);
        sum += z > -INFINITY ? exp(static_cast<double>(z) - top) : 0.0;
      }
      sum = warp_sum(sum);
    }
  }
  __device__ __forceinline__ double operator()(float z) const {
    if constexpr (kSoftmax) return exp(static_cast<double>(z) - top) / sum;
    return 1.0 / (1.0 + exp(-static_cast<double>(z)));
  }
};

// The rank of lane l < count's expert e (numbers rising with the lanes) by its score and
// bias in 64 bits.
template <int DT, bool kSoftmax>
__device__ __noinline__ int rank_exactly(const moe_route_desc& d, const void* row, int e, int count) {
  const int lane = threadIdx.x & 31;
  const ExactScore<DT, kSoftmax> score(row, d.E);
  uint64_t key = 0;
  if (lane < count) key = key_of(score(load_logit<DT>(row, e)) + __ldg(d.bias + e));
  int rank = 0;
  for (int j = 0; j < count; ++j) rank += __shfl_sync(kAll, key, j) + (j < lane) > key;
  return rank;
}

// Which groups stay, as a mask, by their scores and biases in 64 bits.  Lane l < count has
// expert e; among these are the experts that any group counts.
template <int DT, bool kSoftmax>
__device__ __noinline__ uint32_t groups_exactly(const moe_route_desc& d, const void* row, int e, int count) {
  const ExactScore<DT, kSoftmax> score(row, d.E);
  const int lane = threadIdx.x & 31, size = d.E / d.n_group;
  uint64_t key = 0, a = 0, b = 0;
  if (lane < count) key = key_of(score(load_logit<DT>(row, e)) + __ldg(d.bias + e));
  const int g = lane < count ? e / size : -1;
  for (int j = 0; j < count; ++j) {
    const uint64_t k = __shfl_sync(kAll, key, j);
    if (__shfl_sync(kAll, g, j) == lane) {
      b = max(b, min(a, k));
      a = max(a, k);
    }
  }
  if ((d.flags & MOE_ROUTE_GROUP_PAIR) && b != 0) a = key_of(value_of(a) + value_of(b));
  int rank = 0;
  for (int i = 0; i < d.n_group; ++i) rank += __shfl_sync(kAll, a, i) + (i < lane) > a;
  return __ballot_sync(kAll, lane < d.n_group && rank < d.topk_group);
}

}  // namespace
}  // namespace moe
