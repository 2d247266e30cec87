// Routing of many tokens to experts (moe_route): several tokens a warp.
#include <algorithm>

#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kManyWarps = 4;
constexpr int kManyK = 8;           // most experts of a token
constexpr int kManyList = 24;       // most candidates of a token

struct ManyArgs {
  moe_route_desc d;
  int32_t group_lanes;              // of route_exact
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Comparisons, selections and maxima go through a pipe of half the rate, and they are what this
// kernel is made of: so differences and products do where they can.  Values as sortable integers,
// compared and selected, took 37.9 us where these take 33 (65536 tokens of 256 experts).
__device__ __forceinline__ void sort2(float& a, float& b) {      // a the larger
  const float t = fmaxf(a, b);
  b = fminf(a, b);
  a = t;
}
__device__ __forceinline__ void sort4(float* v) {
  sort2(v[0], v[1]);
  sort2(v[2], v[3]);
  sort2(v[0], v[2]);
  sort2(v[1], v[3]);
  sort2(v[1], v[2]);
}
__device__ __forceinline__ void merge4(float* v) {      // a sequence that rises and falls
  sort2(v[0], v[2]);
  sort2(v[1], v[3]);
  sort2(v[0], v[1]);
  sort2(v[2], v[3]);
}
// Of this lane's four and of lane ^ mask's the larger ones (sign 1) or the smaller ones (-1).
template <bool kTurned>
__device__ __forceinline__ void exchange4(float* v, int mask, float sign) {
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __shfl_xor_sync(kAll, v[kTurned ? 3 - i : i], mask);
  const float2 s = make_float2(sign, sign);
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float2 x = __fmul2_rn(make_float2(v[i], v[i + 1]), s), y = __fmul2_rn(make_float2(o[i], o[i + 1]), s);
    const float2 r = __fmul2_rn(make_float2(fmaxf(x.x, y.x), fmaxf(x.y, y.y)), s);
    v[i] = r.x;
    v[i + 1] = r.y;
  }
}
// The sign of a - b behind the bits of m: 1 where a < b (neither of them -0).
__device__ __forceinline__ uint32_t below(uint32_t m, float a, float b) { return __funnelshift_l(__float_as_uint(__fsub_rn(a, b)), m, 1); }

// How many of the earlier lanes' things of L there are, and of all L.
template <int L>
__device__ __forceinline__ int lanes_before(int have, int& all) {
  const int l = threadIdx.x % L;
  int upto = have;
#pragma unroll
  for (int o = 1; o < L; o <<= 1) {
    const int y = __shfl_up_sync(kAll, upto, o, L);
    upto += l >= o ? y : 0;
  }
  all = __shfl_sync(kAll, upto, L - 1, L);
  return upto - have;
}

// L lanes a token, V consecutive experts a lane.
template <int DT, int V, int L>
struct Many {
  static constexpr int kSize = DT == MOE_DTYPE_F32 ? 4 : 2, kVec = 16 / kSize;
  static constexpr int kTokens = 32 / L;
  static constexpr int kPieces = V / kVec, kBiasPieces = V / 4;      // 16 bytes of a lane's logits, biases
  static constexpr int kRuns = V > 8 ? 8 : 4, kRun = V / kRuns;      // of a lane's experts
  static constexpr int kStage = 32 * V * kSize;                      // the logits of a warp's tokens, twice
  static constexpr int kValues = 8 * V * L;                          // of route_exact: over the logits, if they have room
  static constexpr int kScratch = kValues <= kStage ? 0 : kValues;
  // of a token: the values and numbers of the candidates, and the first of their order
  static constexpr int kListLd = 4 * (kManyList + 4), kNumberLd = 2 * kManyList, kSortedLd = kManyK + 2;
  static constexpr int kWarpBytes = 2 * kStage + kScratch + kTokens * (kListLd + kNumberLd + 8 * kSortedLd);
  static constexpr int kSmem = kManyWarps * kWarpBytes + L * V * 4;
  // Where piece j of lane q lies: eight neighbouring lanes that read their j-th ones read
  // all banks.
  static __device__ __forceinline__ int place(int q, int j, int pieces) { return q * pieces + (j ^ (q * pieces / 8 & (pieces - 1))); }
  // the logit of a lane's i-th expert
  static __device__ __forceinline__ float logit(const uint8_t* stage, int q, int i) {
    return load_logit_here(stage + 16 * place(q, i / kVec, kPieces) + kSize * (i % kVec));
  }
  static __device__ __forceinline__ float load_logit_here(const uint8_t* at) {
    if constexpr (DT == MOE_DTYPE_F32) return as_logit(*reinterpret_cast<const float*>(at));
    const uint16_t b = *reinterpret_cast<const uint16_t*>(at);
    return as_logit(DT == MOE_DTYPE_F16 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b));
  }
};

// A warp routes 32 / L tokens at a time, each by L neighbouring lanes: what one lane can do
// alone (scores, the maxima of its experts, its groups') costs as much as in any layout, and
// what lanes have to tell each other is told for several tokens at once.  Rows come through
// shared memory, the next ones while these are routed.
//
// The lanes sort the maxima of their runs of experts; the (k + 1)-th leaves a threshold that at
// least k + 1 experts reach.  These are listed by number, and a lane counts those in front of two
// or three of them.  Neighbours of that order, or the last group that stays and the first that
// does not, that lie too near each other are put in order in 64 bits, by the whole warp.
//
// What bounds it is the pipe of comparisons and the issue of instructions: 65536 tokens of 256
// experts in 8 groups, fp32, take 33 us (2.2 TB/s), 12 with the rows' way through shared memory
// alone, 57 by a warp a token.  Five CTAs an SM: four take 36 us, and six, with the fewer
// registers, 36.
template <int DT, int V, int L, bool kSoftmax>
__global__ void __launch_bounds__(32 * kManyWarps, 5) route_many_kernel(const __grid_constant__ ManyArgs a) {
  using M = Many<DT, V, L>;
  constexpr int kRun = M::kRun, kPer = V * L / 32;
  extern __shared__ __align__(16) uint8_t many_smem[];
  const moe_route_desc& d = a.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L, tok = lane / L, e0 = l * V;
  uint8_t* stage = many_smem + warp * M::kWarpBytes;
  uint8_t* other = stage + M::kStage;
  uint8_t* scratch = other + M::kStage;
  uint8_t* lists = scratch + M::kScratch;
  uint8_t* numbers = lists + M::kTokens * M::kListLd;
  uint2* sorted_all = reinterpret_cast<uint2*>(numbers + M::kTokens * M::kNumberLd);
  float* list = reinterpret_cast<float*>(lists + tok * M::kListLd);
  uint16_t* number = reinterpret_cast<uint16_t*>(numbers + tok * M::kNumberLd);
  uint2* sorted = sorted_all + tok * M::kSortedLd;
  float* bias = reinterpret_cast<float*>(many_smem + kManyWarps * M::kWarpBytes);
  constexpr bool softmax = kSoftmax;
  const bool pair = (d.flags & MOE_ROUTE_GROUP_PAIR) && d.n_group > 1;
  const bool renorm = d.flags & MOE_ROUTE_RENORM, biased = d.bias != nullptr;
  const int stride = d.n_group > 1 ? d.E / d.n_group / V : 1;      // lanes of a group
  const int group = l / stride;
  const bool real = d.n_group == 1 || group < d.n_group;
  const int step = gridDim.x * kManyWarps * M::kTokens, T = static_cast<int>(d.T);

  // experts that are not there: -inf, which no copy writes over
  for (int i = lane; i < 2 * M::kStage / 4; i += 32)
    reinterpret_cast<uint32_t*>(stage)[i] = DT == MOE_DTYPE_F32 ? 0xff800000u : DT == MOE_DTYPE_F16 ? 0xfc00fc00u : 0xff80ff80u;
  grid_dependency_wait();
  grid_launch_dependents();
  auto bias_at = [&](int e) -> float& { return bias[4 * M::place(e / V, e % V / 4, M::kBiasPieces) + e % 4]; };
  if (biased)
    for (int e = threadIdx.x; e < L * V; e += 32 * kManyWarps) {
      const float b = e < d.E ? __ldg(d.bias + e) : 0.0f;
      bias_at(e) = b > -INFINITY ? b : -INFINITY;
    }
  __syncthreads();
  const int limit = d.n_tokens ? max(0, min(*d.n_tokens, T)) : T;
  auto row_of = [&](int t) { return static_cast<const char*>(d.logits) + t * d.logits_ld * M::kSize; };
  const int row_pieces = d.E / M::kVec;
  auto fetch = [&](uint8_t* to, int t0) {
#pragma unroll
    for (int i = 0; i < M::kPieces; ++i) {
      const int at = i * 32 + lane, q = at / M::kPieces, in_row = at % (L * M::kPieces), t = t0 + q / L;
      if (in_row < row_pieces && t < limit)
        cp_async_16(smem_u32(to) + 16 * M::place(q, at % M::kPieces, M::kPieces), row_of(t) + 16 * in_row);
    }
  };
  int t0 = (blockIdx.x * kManyWarps + warp) * M::kTokens;
  fetch(stage, t0);

  for (; t0 < T; t0 += step) {
    const int t = t0 + tok;
    const bool live = t < limit;
    cp_async_wait_all();
    __syncwarp();
    fetch(other, t0 + step);
    float z[V];
#pragma unroll
    for (int j = 0; j < M::kPieces; ++j) {
      const uint4 u = reinterpret_cast<const uint4*>(stage)[M::place(lane, j, M::kPieces)];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MOE_DTYPE_F32) {
          z[4 * j + i] = __uint_as_float(w[i]);
        } else {
          const float2 v = pair_to_float<DT == MOE_DTYPE_F16>(w[i]);
          z[8 * j + 2 * i] = v.x;
          z[8 * j + 2 * i + 1] = v.y;
        }
      }
    }
    float top = 0.0f, sum = 1.0f;
    if (softmax) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, z[i]);      // not of NaN
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      top = fminf(top, FLT_MAX);
      if (!(top > -INFINITY)) top = 0.0f;
      if (biased || !renorm) {               // else nothing asks for the sum
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          z[i] = as_logit(z[i]);
          sum += exp2_fast((z[i] - top) * kLog2e);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (!(sum > 0.0f)) sum = 1.0f;
      }
    }
    // The values, -inf where there is none.  Equal logits and biases give equal bits, here and
    // where a value is made again.
    const float per = rcp_fast(sum), unit = unit_of(softmax, per);
    auto remake = [&](float x, int e, float top, float per) {
      if (!biased) return __fadd_rn(x, 0.0f);
      const float v = softmax ? __fmaf_rn(exp2_fast(__fmul_rn(__fsub_rn(x, top), kLog2e)), per, bias_at(e))
                              : __fadd_rn(rcp_fast(__fadd_rn(exp2_fast(__fmul_rn(x, -kLog2e)), 1.0f)), bias_at(e));
      return x > -INFINITY ? v : -INFINITY;
    };
    float value[V];
    if (biased) {
#pragma unroll
      for (int j = 0; j < M::kBiasPieces; ++j) {
        const float4 b = reinterpret_cast<const float4*>(bias)[M::place(l, j, M::kBiasPieces)];
        const float bs[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          const float2 x = make_float2(z[4 * j + c], z[4 * j + c + 1]), add = make_float2(bs[c], bs[c + 1]);
          float2 v;
          if (softmax) {
            v.x = __fmaf_rn(exp2_fast(__fmul_rn(__fsub_rn(x.x, top), kLog2e)), per, add.x);
            v.y = __fmaf_rn(exp2_fast(__fmul_rn(__fsub_rn(x.y, top), kLog2e)), per, add.y);
          } else {
            const float2 e = __fmul2_rn(x, make_float2(-kLog2e, -kLog2e));
            const float2 s = __fadd2_rn(make_float2(exp2_fast(e.x), exp2_fast(e.y)), make_float2(1.0f, 1.0f));
            v = __fadd2_rn(make_float2(rcp_fast(s.x), rcp_fast(s.y)), add);
          }
          value[4 * j + c] = x.x > -INFINITY ? v.x : -INFINITY;
          value[4 * j + c + 1] = x.y > -INFINITY ? v.y : -INFINITY;
        }
      }
    } else {
      // logits as they are, but -0 as 0: the difference of the two has a sign
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 v = __fadd2_rn(make_float2(as_logit(z[i]), as_logit(z[i + 1])), make_float2(0.0f, 0.0f));
        value[i] = v.x;
        value[i + 1] = v.y;
      }
    }
    // the maxima of the lane's runs
    float run[M::kRuns], best = -INFINITY, second = -INFINITY;
    if (pair) {
#pragma unroll
      for (int r = 0; r < M::kRuns; ++r) {
        float low = -INFINITY;
#pragma unroll
        for (int i = 0; i < kRun; i += 2) {
          const float x = value[r * kRun + i], y = value[r * kRun + i + 1], h = fmaxf(x, y), s = fminf(x, y);
          low = i ? fmaxf(fmaxf(low, s), fminf(run[r], h)) : s;
          run[r] = i ? fmaxf(run[r], h) : h;
        }
        second = fmaxf(fmaxf(second, low), fminf(best, run[r]));
        best = fmaxf(best, run[r]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < M::kRuns; ++r) {
        run[r] = value[r * kRun];
#pragma unroll
        for (int i = 1; i < kRun; ++i) run[r] = fmaxf(run[r], value[r * kRun + i]);
        best = fmaxf(best, run[r]);
      }
    }
    // groups
    bool kept = real;
    uint32_t doubt = 0;                        // lanes of tokens that route_exact decides
    if (d.n_group > 1) {
#pragma unroll 1
      for (int o = stride / 2; o > 0; o >>= 1) {
        const float ob = __shfl_xor_sync(kAll, best, o), os = __shfl_xor_sync(kAll, second, o);
        second = fmaxf(fminf(best, ob), fmaxf(second, os));
        best = fmaxf(best, ob);
      }
      const float mark = pair && second > -INFINITY ? best + second : best;
      int rank = 0;
      float next = -INFINITY;                  // the mark behind this group's
#pragma unroll 4
      for (int g = 0; g < d.n_group; ++g) {
        const float x = __shfl_sync(kAll, mark, g * stride, L);
        const bool front = x > mark || (x == mark && g < group);
        rank += front;
        next = fmaxf(next, front || g == group ? -INFINITY : x);
      }
      kept = real && rank < d.topk_group;
      if (biased) {
        const bool near = live && real && rank == d.topk_group - 1 && next > -INFINITY &&
                          !(mark - next > 4.0f * near_of(mark, unit));
        uint32_t again = __ballot_sync(kAll, near);
        if (again) {
          // the experts that a group may count, up to 32, settle it in 64 bits
          const float v = pair && second > -INFINITY ? second : best, from = v <= FLT_MAX ? v - 4.0f * near_of(v, unit) : v;
          uint32_t reach = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) reach |= value[i] > -INFINITY && value[i] >= from ? 1u << i : 0u;
          int all, at = lanes_before<L>(__popc(reach), all), *among = reinterpret_cast<int*>(lists);
          while (again) {
            const int which = (__ffs(again) - 1) / L, n = __shfl_sync(kAll, all, which * L);
            const uint32_t its = ((1u << L) - 1) << which * L;
            again &= ~its;
            if (n > 32) {
              doubt |= its;
              continue;
            }
            if (tok == which)
              for (; reach; reach &= reach - 1) among[at++] = e0 + __ffs(reach) - 1;
            __syncwarp();
            const char* row = row_of(t0 + which);
            const int e = lane < n ? among[lane] : 0;
            const uint32_t groups = groups_exactly<DT, kSoftmax>(d, row, e, n);
            if (tok == which) kept = real && ((groups >> group) & 1);
            __syncwarp();
          }
        }
      }
    }
    kept = kept && live;
    // the threshold
    float least;
    {
      sort4(run);
      if constexpr (M::kRuns == 8) {           // the four largest of the eight
        sort4(run + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) run[i] = fmaxf(run[i], run[7 - i]);
        merge4(run);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) run[i] = kept ? run[i] : -INFINITY;
      // two lanes' fours to one order, then two pairs' and so on (K. E. Batcher's bitonic merging)
#pragma unroll
      for (int w = 1; w < L; w *= 2) {
        exchange4<true>(run, 2 * w - 1, l & w ? -1.0f : 1.0f);
#pragma unroll
        for (int h = w / 2; h > 0; h /= 2) exchange4<false>(run, h, l & h ? -1.0f : 1.0f);
        merge4(run);
      }
      const float it = d.k & 2 ? (d.k & 1 ? run[3] : run[2]) : (d.k & 1 ? run[1] : run[0]);
      least = fmaxf(__shfl_sync(kAll, it, d.k / 4, L), -FLT_MAX);
    }
    // the experts that reach it, in the order of their numbers
    uint32_t reach = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) reach = below(reach, value[i], least);
    reach = kept ? ~reach & (V < 32 ? (1u << V % 32) - 1 : kAll) : 0u;
    int count;
    const int before = lanes_before<L>(__popc(reach), count);
    const bool many = count > kManyList;
    for (int at = before; reach; reach &= reach - 1, ++at)
      if (at < kManyList) number[at] = static_cast<uint16_t>(e0 + __ffs(reach) - 1);
    for (int i = l; i < M::kSortedLd / 2; i += L) reinterpret_cast<uint4*>(sorted)[i] = make_uint4(0u, kAll, 0u, kAll);
    __syncwarp();
    const int longest = __reduce_max_sync(kAll, many ? 0 : count);
    for (int at = l; at < kManyList && at - l < longest; at += L) {
      const int e = at < count ? number[at] : 0;
      list[at] = at < count ? remake(M::logit(stage, tok * L + e / V, e % V), e, top, per) : -INFINITY;
    }
    __syncwarp();
    for (int at = l; at < longest; at += 2 * L) {
      const float x = list[at], y = at + L < kManyList && at - l + L < longest ? list[at + L] : -INFINITY;
      uint32_t front_x = 0, front_y = 0;
#pragma unroll 1
      for (int j = 0; j < longest; j += 4) {
        const float4 o = *reinterpret_cast<const float4*>(list + j);
        front_x = below(below(below(below(front_x, x, o.x), x, o.y), x, o.z), x, o.w);
        front_y = below(below(below(below(front_y, y, o.x), y, o.y), y, o.z), y, o.w);
      }
      const int rank_x = __popc(front_x), rank_y = __popc(front_y);
      if (!many && x > -INFINITY && rank_x <= d.k) sorted[rank_x] = make_uint2(__float_as_uint(x), number[at]);
      if (!many && y > -INFINITY && rank_y <= d.k) sorted[rank_y] = make_uint2(__float_as_uint(y), number[at + L]);
    }
    __syncwarp();
    // equal values leave a place empty: the lowest number first
    const int places = many ? 0 : min(count, d.k + 1);
    if (__any_sync(kAll, (l < places && sorted[l].y == kAll) || (l + 1 < places && sorted[l + 1].y == kAll))) {
      if (!many)
        for (int at = l; at < count; at += L) {
          const float x = list[at];
          int rank = 0;
          for (int j = 0; j < count; ++j) rank += list[j] > x || (list[j] == x && j < at);
          if (rank <= d.k) sorted[rank] = make_uint2(__float_as_uint(x), number[at]);
        }
    }
    // values of the groups that stay, for what the warp does together
    const uint32_t open = __ballot_sync(kAll, kept);
    auto value_of_expert = [&](int first, int e, float top, float per) {
      const int q = first + e / V;
      return (open >> q) & 1 ? remake(M::logit(stage, q, e % V), e, top, per) : -INFINITY;
    };
    for (uint32_t full = __ballot_sync(kAll, many && l == 0); full; full &= full - 1) {
      // more candidates than the list holds: the largest one after another, by the warp
      const int first = __ffs(full) - 1;
      const float its_top = __shfl_sync(kAll, top, first), its_per = __shfl_sync(kAll, per, first);
      uint32_t x[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float v = value_of_expert(first, i * 32 + lane, its_top, its_per);
        x[i] = v > -INFINITY ? key_of(v) : 0u;
      }
#pragma unroll 1
      for (int j = 0; j <= d.k; ++j) {
        uint32_t m = 0;
        int e = INT32_MAX;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (x[i] > m) {
            m = x[i];
            e = i * 32 + lane;
          }
        const uint32_t most = __reduce_max_sync(kAll, m);
        e = __reduce_min_sync(kAll, m == most ? e : INT32_MAX);
        if (lane == 0) sorted_all[first / L * M::kSortedLd + j] = make_uint2(__float_as_uint(value_of(most)), e);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (e == i * 32 + lane) x[i] = 0;
      }
    }
    __syncwarp();
    uint2 it = l < d.k ? sorted[l] : make_uint2(0u, kAll);
    bool lost = false;                         // the logits are written over
    if (biased) {
      const uint2 next = l < d.k ? sorted[l + 1] : make_uint2(0u, kAll);
      const float v = __uint_as_float(it.x);
      const bool near = next.y != kAll && !(v - __uint_as_float(next.x) > near_of(v, unit));
      uint32_t again = __ballot_sync(kAll, near) & ~doubt;
      if (again | doubt) {
        while (again) {
          const int which = (__ffs(again) - 1) / L, first = which * L, n = __shfl_sync(kAll, count, first);
          const uint32_t its = ((1u << L) - 1) << first;
          again &= ~its;
          doubt |= its;
          // the experts that may be among the k, up to 32
          const float kth = __uint_as_float(sorted_all[which * M::kSortedLd + min(d.k, n) - 1].x), at_least = kth - near_of(kth, __shfl_sync(kAll, unit, first));
          const float its_top = __shfl_sync(kAll, top, first), its_per = __shfl_sync(kAll, per, first);
          uint32_t may = 0;
          for (int i = 0; i < kPer; ++i) {
            const float x = value_of_expert(first, lane * kPer + i, its_top, its_per);
            may |= x > -INFINITY && !(x < at_least) ? 1u << i : 0u;
          }
          int all, at = lanes_before<32>(__popc(may), all), *among = reinterpret_cast<int*>(lists);
          if (all > 32) continue;
          for (; may; may &= may - 1) among[at++] = lane * kPer + __ffs(may) - 1;
          __syncwarp();
          const char* row = row_of(t0 + which);
          const int e = lane < all ? among[lane] : 0, rank = rank_exactly<DT, kSoftmax>(d, row, e, all);
          if (lane < all && rank < d.k) sorted_all[which * M::kSortedLd + rank] = make_uint2(0u, e);
          __syncwarp();
          doubt &= ~its;
        }
        lost = doubt && M::kScratch == 0;
        while (doubt) {
          const int which = (__ffs(doubt) - 1) / L;
          doubt &= ~(((1u << L) - 1) << which * L);
          const int id = route_exact<DT>(d, row_of(t0 + which), reinterpret_cast<uint64_t*>(M::kScratch ? scratch : stage), a.group_lanes);
          if (lane < d.k) sorted_all[which * M::kSortedLd + lane] = make_uint2(0u, id);
          __syncwarp();
        }
        if (l < d.k) it = sorted[l];
      }
    }
    const bool chosen = live && it.y != kAll;
    const int expert = chosen ? static_cast<int>(it.y) : -1;
    float x = -INFINITY;
    if (chosen) x = lost ? load_logit<DT>(row_of(t), expert) : M::logit(stage, tok * L + expert / V, expert % V);
    float s = 0.0f;
    if (softmax) {
      // shares of each other do not depend on what was not chosen, and not underflow beside it
      float base = top;
      if (renorm) {
        base = x;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) base = fmaxf(base, __shfl_xor_sync(kAll, base, o));
        base = fmaxf(base, -FLT_MAX);
      }
      s = __fdividef(expf(x - base), renorm ? 1.0f : sum);
    } else if (chosen) {
      // from the exponential that is at most 1: down to subnormal scores
      const float u = expf(-fabsf(x));
      s = __fdividef(x < 0.0f ? u : 1.0f, 1.0f + u);
    }
    if (renorm) {
      float all = s;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) all += __shfl_xor_sync(kAll, all, o);
      if constexpr (!softmax) {
        const bool small = all < 0x1p-30f;     // of which fp32 may have few bits, or none
        if (__any_sync(kAll, small && chosen)) {
          float base = x, sum_of = 0.0f;
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) base = fmaxf(base, __shfl_xor_sync(kAll, base, o));
          const float share = sum_of = small_score(x, base);
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) sum_of += __shfl_xor_sync(kAll, sum_of, o);
          if (small) {
            s = share;
            all = fmaxf(sum_of, FLT_MIN);
          }
        }
      }
      s = __fdividef(s, all);
    }
    if (l < d.k && t < T) {
      d.topk_ids[t * d.ids_ld + l] = expert;
      d.topk_w[t * d.w_ld + l] = chosen ? s * d.scale : 0.0f;
    }
    __syncwarp();
    if (lost && d.E < L * V) {                 // what no copy writes
      for (int i = lane; i < M::kStage / 4; i += 32)
        reinterpret_cast<uint32_t*>(stage)[i] = DT == MOE_DTYPE_F32 ? 0xff800000u : DT == MOE_DTYPE_F16 ? 0xfc00fc00u : 0xff80ff80u;
      __syncwarp();
    }
    uint8_t* was = stage;
    stage = other;
    other = was;
  }
  cp_async_wait_all();
}

// Lanes of a token and experts of a lane, for E experts.
int experts_of_lane(int E) { return E <= 64 ? 8 : E <= 128 ? 16 : 32; }

template <int DT, int V, int L, bool kSoftmax>
int launch_many(const ManyArgs& a, cudaStream_t st) {
  using M = Many<DT, V, L>;
  const int64_t batch = kManyWarps * M::kTokens;
  const int64_t ctas = std::min<int64_t>((a.d.T + batch - 1) / batch, 5ll * num_sms());
  return launch_pdl(route_many_kernel<DT, V, L, kSoftmax>, dim3(static_cast<unsigned>(ctas)), dim3(32 * kManyWarps), M::kSmem, st, a);
}

template <int DT, bool kSoftmax>
int pick_many(const ManyArgs& a, cudaStream_t st) {
  if (a.d.E <= 64) return launch_many<DT, 8, 8, kSoftmax>(a, st);
  if (a.d.E <= 128) return launch_many<DT, 16, 8, kSoftmax>(a, st);
  if (a.d.E <= 256) return launch_many<DT, 32, 8, kSoftmax>(a, st);
  return launch_many<DT, 32, 16, kSoftmax>(a, st);
}

template <int DT>
int pick_many(const ManyArgs& a, cudaStream_t st) {
  return a.d.flags & MOE_ROUTE_SOFTMAX ? pick_many<DT, true>(a, st) : pick_many<DT, false>(a, st);
}

}  // namespace

bool is_for_route_many(const moe_route_desc& d) {
  const int64_t bytes = d.dtype == MOE_DTYPE_F32 ? 4 : 2;
  const int V = experts_of_lane(d.E), size = d.E / d.n_group;
  // Enough tokens for all warps, at this many a warp: 8192 tokens of 256 experts in groups take
  // 9.3 us here and 10.2 by a warp a token, 4096 take 7.5 and 6.8; 4096 of 512 take 10.9 and 23.8.
  // (What is refused here goes by a warp a token: 65536 tokens of 512 experts, 10 each, 105 us; of 160
  // in 8 groups of 20, 4 of which stay, 84.)
  if (d.T < (d.E <= 256 ? 8192 : 4096) || d.E > 512 || d.k > kManyK) return false;
  // rows in pieces of 16 bytes
  if (reinterpret_cast<uintptr_t>(d.logits) % 16 || d.logits_ld * bytes % 16 || d.E * bytes % 16) return false;
  // groups of whole lanes, by the values that rank
  if (d.n_group > 1 && (size % V || (size / V & (size / V - 1)) || (d.bias == nullptr && (d.flags & MOE_ROUTE_GROUP_PAIR)))) return false;
  // runs enough for a threshold that few experts reach
  return 5 * (d.k + 1) <= 3 * (4 * d.topk_group * size / V);
}

int route_many(const moe_route_desc& d, int group_lanes, cudaStream_t st) {
  const ManyArgs a{d, group_lanes};
  if (d.dtype == MOE_DTYPE_F32) return pick_many<MOE_DTYPE_F32>(a, st);
  return d.dtype == MOE_DTYPE_F16 ? pick_many<MOE_DTYPE_F16>(a, st) : pick_many<MOE_DTYPE_BF16>(a, st);
}

}  // namespace moe
