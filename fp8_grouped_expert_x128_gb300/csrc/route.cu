// Routing to experts: softmax or sigmoid scores, a bias for balance, groups,
// top-k, renormalised weights (moe_route).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kRouteWarps = 4;      // tokens of a CTA, a warp each
constexpr uint32_t kAll = 0xffffffffu;

struct RouteArgs {
  moe_route_desc d;
  int32_t wide;          // a lane's logits (its biases) in one or more aligned loads
  int32_t wide_bias;
  int32_t slot;          // shared memory of a warp, 8-byte units
  int32_t group_lanes;
};

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
// its sum is off by less than 2^-19 of it, by which two of them shift together.  Adding a bias
// rounds either to 2^-24.
__device__ __forceinline__ float near_of(float v, bool softmax) { return (softmax ? 0x1p-18f : 0x1p-20f) + 0x1p-22f * fabsf(v); }

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

// VPL consecutive values of a lane, from e0 = lane * VPL on; `rest` past the last.
template <int DT, int VPL>
__device__ __forceinline__ void load_lane(const void* row, int E, bool wide, float rest, float (&z)[VPL]) {
  constexpr int kSize = DT == MOE_DTYPE_F32 ? 4 : 2, kBytes = VPL * kSize;
  const int e0 = (threadIdx.x & 31) * VPL;
  if (wide && e0 + VPL <= E) {
    const char* at = static_cast<const char*>(row) + static_cast<size_t>(e0) * kSize;
    uint32_t w[(kBytes + 3) / 4];
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(at) + i);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(at));
      w[0] = u.x;
      w[1] = u.y;
    } else if constexpr (kBytes == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(at));
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if constexpr (DT == MOE_DTYPE_F32) {
        z[i] = __uint_as_float(w[i]);
      } else {
        const uint16_t h = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        z[i] = DT == MOE_DTYPE_F16 ? __half2float(__ushort_as_half(h)) : bf16_bits_to_float(h);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) z[i] = e0 + i < E ? raw_logit<DT>(row, e0 + i) : rest;
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// For the few tokens whose candidates the list does not hold: the `most` largest of E keys in
// shared memory one after another.  Returns how many there are.
__device__ __noinline__ int select_slowly(uint32_t* key, int E, int most, uint2* list) {
  const int lane = threadIdx.x & 31;
  int count = 0;
  for (; count < most; ++count) {
    uint32_t m = 0;
    int n = INT32_MAX;
    for (int e = lane; e < E; e += 32)
      if (key[e] > m) {
        m = key[e];
        n = e;
      }
    const uint32_t first = __reduce_max_sync(kAll, m);
    if (first == 0) break;
    n = __reduce_min_sync(kAll, m == first ? n : INT32_MAX);
    if (lane == (n & 31)) {
      key[n] = 0;
      list[count] = make_uint2(first, n);
    }
    __syncwarp();
  }
  return count;
}

// The rank of lane l < count's expert e (numbers rising with the lanes) by its sigmoid and
// bias in 64 bits.
template <int DT>
__device__ __noinline__ int rank_exactly(const void* row, const float* bias, int e, int count) {
  const int lane = threadIdx.x & 31;
  uint64_t key = 0;
  if (lane < count) key = key_of(1.0 / (1.0 + exp(-static_cast<double>(load_logit<DT>(row, e)))) + __ldg(bias + e));
  int rank = 0;
  for (int j = 0; j < count; ++j) rank += __shfl_sync(kAll, key, j) + (j < lane) > key;
  return rank;
}

// Which groups stay, as a mask, by their sigmoids and biases in 64 bits.  Lane l < count has
// expert e; among these are the experts that any group counts.
template <int DT>
__device__ __noinline__ uint32_t groups_exactly(const moe_route_desc& d, const void* row, int e, int count) {
  const int lane = threadIdx.x & 31, size = d.E / d.n_group;
  uint64_t key = 0, a = 0, b = 0;
  if (lane < count) key = key_of(1.0 / (1.0 + exp(-static_cast<double>(load_logit<DT>(row, e)))) + __ldg(d.bias + e));
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

// How many of the earlier lanes' things there are, and of all.
__device__ __forceinline__ int lanes_before(int have, int& all) {
  const int lane = threadIdx.x & 31;
  int upto = have;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, upto, o);
    upto += lane >= o ? y : 0;
  }
  all = __shfl_sync(kAll, upto, 31);
  return upto - have;
}

// A warp routes one token after another, in fp32 as far as that decides.  What bounds it is
// the number of instructions (256 experts: 40 instructions' time of loads, some 450 of
// arithmetic and exchange a token), so values become sortable keys once, and selection works
// on few of them: the k + 1 largest of the lanes' maxima leave a threshold that at least k + 1
// experts reach and seldom many more.  These (32 at most) go to a lane each, in the order of
// their numbers, which counts those in front of it.  Where two neighbours of that order, or
// the last group that stays and the first that does not, lie too near, the token is decided
// in 64 bits.
template <int DT, int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps, VPL <= 8 ? 8 : 2) route_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ uint64_t route_smem[];
  const moe_route_desc& d = a.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * VPL;
  constexpr int kSize = DT == MOE_DTYPE_F32 ? 4 : 2;
  uint64_t* wide = route_smem + static_cast<size_t>(warp) * a.slot;
  uint2* list = reinterpret_cast<uint2*>(wide);               // 33 and 3 of padding
  uint32_t* sorted = reinterpret_cast<uint32_t*>(wide + 36);  // 34
  const bool softmax = d.flags & MOE_ROUTE_SOFTMAX, pair = (d.flags & MOE_ROUTE_GROUP_PAIR) && d.n_group > 1;
  const bool renorm = d.flags & MOE_ROUTE_RENORM, biased = d.bias != nullptr;
  const int size = d.E / d.n_group;
  // lanes of a group, if groups are whole lanes
  const bool whole = size % VPL == 0 && (size / VPL & (size / VPL - 1)) == 0;
  const int stride = whole ? size / VPL : a.group_lanes, mine = lane / stride;
  const bool real = mine < d.n_group;
  grid_dependency_wait();
  grid_launch_dependents();
  const int step = gridDim.x * kRouteWarps, T = static_cast<int>(d.T);
  const int limit = d.n_tokens ? max(0, min(*d.n_tokens, T)) : T;
  auto row_of = [&](int t) { return static_cast<const char*>(d.logits) + t * d.logits_ld * kSize; };
  int t = blockIdx.x * kRouteWarps + warp;
  float bias[VPL], next[VPL];
  if (biased) load_lane<MOE_DTYPE_F32, VPL>(d.bias, d.E, a.wide_bias, 0.0f, bias);
  if (t < limit) load_lane<DT, VPL>(row_of(t), d.E, a.wide, -INFINITY, next);

  for (; t < T; t += step) {
    if (t >= limit) {
      if (lane < d.k) {
        d.topk_ids[t * d.ids_ld + lane] = -1;
        d.topk_w[t * d.w_ld + lane] = 0.0f;
      }
      continue;
    }
    const char* row = row_of(t);
    float z[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) z[i] = next[i];
    if (t + step < limit) load_lane<DT, VPL>(row_of(t + step), d.E, a.wide, -INFINITY, next);

    float top = 0.0f, sum = 1.0f;
    if (softmax) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) top = fmaxf(top, z[i]);      // not of NaN
      top = fminf(warp_max(top), FLT_MAX);
      if (!(top > -INFINITY)) top = 0.0f;
      if (biased || pair || !renorm) {         // else nothing asks for the sum
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          z[i] = z[i] > -INFINITY ? fminf(z[i], FLT_MAX) : -INFINITY;
          sum += exp2_fast((z[i] - top) * kLog2e);
        }
        sum = warp_sum(sum);
        if (!(sum > 0.0f)) sum = 1.0f;
      }
    }
    // keys of the values.  Equal logits and biases give equal bits.
    uint32_t key[VPL];
    const float per = rcp_fast(sum);
    if (biased) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float v = softmax ? __fmaf_rn(exp2_fast((z[i] - top) * kLog2e), per, bias[i])
                                : __fadd_rn(rcp_fast(__fadd_rn(exp2_fast(z[i] * -kLog2e), 1.0f)), bias[i]);
        key[i] = z[i] > -INFINITY && v > -INFINITY ? key_of_sum(v) : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = z[i] > -INFINITY ? key_of(fminf(z[i], FLT_MAX)) : 0u;
    }
    bool unsure = false;
    if (d.n_group > 1) {
      uint32_t best = 0, second = 0;        // of the lane's experts, and then of its group's
      const bool scores = pair && !biased;
      if (whole && !scores) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
        if (pair) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < VPL; ++i) {
            second = max(second, min(m, key[i]));
            m = max(m, key[i]);
          }
        }
      } else {
        // groups that end inside a lane, or that count scores where logits rank: as many lanes
        // as there are for each group, over shared memory
        uint32_t* v = reinterpret_cast<uint32_t*>(wide);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (e0 + i < d.E) {
            const float x = fminf(z[i], FLT_MAX);
            v[e0 + i] = key[i] == 0 || !scores ? key[i]
                        : key_of(softmax ? exp2_fast((x - top) * kLog2e) * per : rcp_fast(exp2_fast(x * -kLog2e) + 1.0f));
          }
        __syncwarp();
        if (real)
          for (int j = lane % stride; j < size; j += stride) {
            const uint32_t x = v[mine * size + j];
            second = max(second, min(best, x));
            best = max(best, x);
          }
        __syncwarp();
      }
#pragma unroll 1
      for (int o = stride / 2; o > 0; o >>= 1) {
        const uint32_t ob = __shfl_xor_sync(kAll, best, o), os = __shfl_xor_sync(kAll, second, o);
        second = max(min(best, ob), max(second, os));
        best = max(best, ob);
      }
      const uint32_t mark = !real ? 0u : pair && second ? key_of_sum(value_of(best) + value_of(second)) : best;
      // the largest marks one after another; where some are equal, or groups without an open
      // expert stay, by their ranks
      uint32_t rest = mark, low = 0;
#pragma unroll 1
      for (int j = 0; j < d.topk_group; ++j) {
        low = __reduce_max_sync(kAll, rest);
        rest = rest == low ? 0u : rest;
      }
      const uint32_t out = __reduce_max_sync(kAll, rest);
      bool kept = mark > out;
      if (low == 0 || __popc(__ballot_sync(kAll, kept)) != d.topk_group * stride) {
        int rank = 0;
        for (int g = 0; g < d.n_group; ++g) rank += __shfl_sync(kAll, mark, g * stride) + (g < mine) > mark;
        kept = real && rank < d.topk_group;
        if (biased || pair) {
          low = __reduce_min_sync(kAll, kept && mark ? mark : 0xffffffffu);
          const uint32_t next_one = __reduce_max_sync(kAll, real && !kept ? mark : 0u);
          unsure = next_one && !(value_of(low) - value_of(next_one) > 4.0f * near_of(value_of(low), softmax));
        }
      } else if (biased || pair) {
        unsure = out && !(value_of(low) - value_of(out) > 4.0f * near_of(value_of(low), softmax));
      }
      if (unsure && whole && biased && !softmax) {
        // the experts that a group may count, up to a lane each, settle it in 64 bits
        const float v = value_of(pair && second ? second : best);
        const uint32_t from = best ? key_of(v - 4.0f * near_of(v, false)) : 0xffffffffu;
        int have = 0, count;
#pragma unroll
        for (int i = 0; i < VPL; ++i) have += key[i] >= from;
        int at = lanes_before(have, count);
        if (count <= 32) {
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (key[i] >= from) sorted[at++] = e0 + i;
          __syncwarp();
          kept = real && ((groups_exactly<DT>(d, row, lane < count ? sorted[lane] : 0, count) >> mine) & 1);
          unsure = false;
          __syncwarp();
        }
      }
      if (whole) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = kept ? key[i] : 0u;
      } else {
        const uint32_t groups = __ballot_sync(kAll, kept && lane % stride == 0);
        int g = e0 / size, left = size - e0 % size;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (g >= d.n_group || !((groups >> (g * stride)) & 1)) key[i] = 0u;
          if (--left == 0) {
            ++g;
            left = size;
          }
        }
      }
    }
    // the threshold
    uint32_t most = key[0], least = 1;
#pragma unroll
    for (int i = 1; i < VPL; ++i) most = max(most, key[i]);
    if constexpr (VPL > 1) {
#pragma unroll 4
      for (int j = 0; j <= d.k; ++j) {
        least = __reduce_max_sync(kAll, most);
        most = most == least ? 0u : most;
      }
      least = max(least, 1u);
    }
    // the experts that reach it, a lane each, in the order of their numbers
    int have = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) have += key[i] >= least;
    int count, rank = lane;
    const int first = lanes_before(have, count);
    const bool few = count <= 32;
    uint2 me = make_uint2(0u, 0u);
    if (few) {
      uint2* at = list + first;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (key[i] >= least) *at++ = make_uint2(key[i], e0 + i);
      if (lane < 3) list[count + lane] = make_uint2(0u, 0u);
      __syncwarp();
      if (lane < count) me = list[lane];
      rank = 0;
#pragma unroll 1
      for (int j = 0; j < count; j += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(list + j), y = *reinterpret_cast<const uint4*>(list + j + 2);
        rank += (x.x > me.x) + (x.z > me.x) + (y.x > me.x) + (y.z > me.x);
      }
      if (__reduce_add_sync(kAll, lane < count ? rank : 0) != count * (count - 1) / 2)      // equal keys: the lowest number first
        for (int j = 0; j < count; ++j) rank += list[j].x == me.x && j < lane;
    } else {
      uint32_t* all = reinterpret_cast<uint32_t*>(wide + 54);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e0 + i < d.E) all[e0 + i] = key[i];
      __syncwarp();
      count = select_slowly(all, d.E, d.k + 1, list);
      if (lane < count) me = list[lane];
      if (lane == 0 && count == 33) sorted[32] = list[32].x;
    }
    if (biased) {
      if (lane < count) sorted[rank] = me.x;
      __syncwarp();
      const bool judged = lane < count && rank < d.k && rank + 1 < count;
      const float v = value_of(me.x);
      if (__any_sync(kAll, judged && !(v - value_of(sorted[rank + 1]) > near_of(v, softmax)))) {
        // where the k-th is clear of what stayed below the threshold, the listed experts settle
        // it among themselves (but for a softmax, whose sum would take all of them)
        const float kth = value_of(sorted[min(d.k, count) - 1]);
        if (!softmax && few && (least == 1u || kth - value_of(least) > near_of(kth, false)))
          rank = rank_exactly<DT>(row, d.bias, me.y, count);
        else
          unsure = true;
      }
    }
    if (unsure) {
      __syncwarp();
      const int id = route_exact<DT>(d, row, wide, a.group_lanes);
      count = __popc(__ballot_sync(kAll, id >= 0));
      me.y = id;
      rank = lane;
    }
    const bool chosen = lane < count && rank < d.k;
    float s = 0.0f;
    if (softmax) {
      const float x = chosen ? load_logit<DT>(row, me.y) : -INFINITY;
      // shares of each other do not depend on what was not chosen, and not underflow beside it
      const float from = renorm ? fmaxf(warp_max(x), -FLT_MAX) : top;
      s = __fdividef(expf(x - from), renorm ? 1.0f : sum);
    } else if (chosen) {
      // from the exponential that is at most 1: down to subnormal scores
      const float x = load_logit<DT>(row, me.y), u = expf(-fabsf(x));
      s = __fdividef(x < 0.0f ? u : 1.0f, 1.0f + u);
    }
    if (renorm) {
      const float all = warp_sum(s), up = all < 0x1p-60f ? 0x1p100f : 1.0f;
      s = all > 0.0f ? __fdividef(s * up, all * up) : 0.0f;
    }
    int32_t* ids = d.topk_ids + t * d.ids_ld;
    float* weights = d.topk_w + t * d.w_ld;
    if (chosen) {
      ids[rank] = static_cast<int32_t>(me.y);
      weights[rank] = s * d.scale;
    } else if (lane >= count && lane < d.k) {
      ids[lane] = -1;
      weights[lane] = 0.0f;
    }
    __syncwarp();
  }
}

template <int DT, int VPL>
int launch_route(RouteArgs& a, cudaStream_t st) {
  constexpr int kSize = DT == MOE_DTYPE_F32 ? 4 : 2;
  const int64_t unit = std::min(16, VPL * kSize);
  a.wide = reinterpret_cast<uintptr_t>(a.d.logits) % unit == 0 && a.d.logits_ld * kSize % unit == 0;
  a.wide_bias = reinterpret_cast<uintptr_t>(a.d.bias) % std::min(16, VPL * 4) == 0;
  a.slot = 54 + a.d.E;                            // the lists and all keys, or 64-bit values
  a.group_lanes = 1;
  while (2 * a.group_lanes * a.d.n_group <= 32) a.group_lanes *= 2;
  // a few tokens a warp, so that a row is on its way while another is routed
  const int64_t ctas = std::min<int64_t>((a.d.T + kRouteWarps - 1) / kRouteWarps, 32ll * num_sms());
  return launch_pdl(route_kernel<DT, VPL>, dim3(static_cast<unsigned>(ctas)), dim3(32 * kRouteWarps),
                    sizeof(uint64_t) * kRouteWarps * a.slot, st, a);
}

template <int DT>
int pick_route(RouteArgs& a, cudaStream_t st) {
  if (a.d.E <= 32) return launch_route<DT, 1>(a, st);
  if (a.d.E <= 64) return launch_route<DT, 2>(a, st);
  if (a.d.E <= 128) return launch_route<DT, 4>(a, st);
  if (a.d.E <= 256) return launch_route<DT, 8>(a, st);
  if (a.d.E <= 512) return launch_route<DT, 16>(a, st);
  return launch_route<DT, 32>(a, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_route(const moe_route_desc* d, void* stream) {
  MOE_CHECK_ARG(d != nullptr);
  MOE_CHECK_ARG((d->flags & ~(MOE_ROUTE_SOFTMAX | MOE_ROUTE_RENORM | MOE_ROUTE_GROUP_PAIR)) == 0);
  MOE_CHECK_ARG(d->dtype == MOE_DTYPE_BF16 || d->dtype == MOE_DTYPE_F16 || d->dtype == MOE_DTYPE_F32);
  MOE_CHECK_ARG(d->T >= 0 && d->E >= 1 && d->E <= 1024 && d->k >= 1 && d->k <= 32 && std::isfinite(d->scale));
  MOE_CHECK_ARG(d->n_group >= 1 && d->E % d->n_group == 0 && d->topk_group >= 1 && d->topk_group <= d->n_group);
  MOE_CHECK_ARG(d->k <= d->topk_group * (d->E / d->n_group));
  MOE_CHECK_ARG(d->logits_ld >= d->E && d->ids_ld >= d->k && d->w_ld >= d->k);
  if (d->n_group > 32 || d->T > (1 << 24) || d->logits_ld > INT32_MAX || d->ids_ld > INT32_MAX || d->w_ld > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (d->T == 0) return MOE_OK;
  MOE_CHECK_ARG(d->logits && d->topk_ids && d->topk_w);
  const uintptr_t unit = d->dtype == MOE_DTYPE_F32 ? 3 : 1;
  MOE_CHECK_ARG((reinterpret_cast<uintptr_t>(d->logits) & unit) == 0 && (reinterpret_cast<uintptr_t>(d->topk_ids) & 3) == 0 &&
                (reinterpret_cast<uintptr_t>(d->topk_w) & 3) == 0 && (reinterpret_cast<uintptr_t>(d->bias) & 3) == 0 &&
                (reinterpret_cast<uintptr_t>(d->n_tokens) & 3) == 0);
  if (int rc = check_device()) return rc;
  RouteArgs a{*d, 0, 0, 0, 0};
  if (d->dtype == MOE_DTYPE_F32) return pick_route<MOE_DTYPE_F32>(a, as_stream(stream));
  return d->dtype == MOE_DTYPE_F16 ? pick_route<MOE_DTYPE_F16>(a, as_stream(stream)) : pick_route<MOE_DTYPE_BF16>(a, as_stream(stream));
}
