// Routing to experts: softmax or sigmoid scores, a bias for balance, groups,
// top-k, renormalised weights (moe_route).
#include <algorithm>
#include <utility>

#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kRouteWarps = 4;      // tokens of a CTA, a warp each

struct RouteArgs {
  moe_route_desc d;
  int32_t wide;          // a lane's logits (its biases) in one or more aligned loads
  int32_t wide_bias;
  int32_t slot;          // shared memory of a warp, 8-byte units
  int32_t group_lanes;
};

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

// For tokens whose candidates the list does not hold: the `most` largest of E keys in shared memory
// one after another.  Returns how many there are.  Few come here while the groups that stay span more
// than k lanes.  Where they span fewer, the lanes' maxima give no threshold and every token does:
// 1024 tokens of 256 experts, 8 of 2 of 8 groups, take 27 us (of 4 groups 5.3), 16 of 4 groups 40, 24
// without groups 37.
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

// A lane's share of the chosen scores, where fp32 has few bits of these or none.
template <int DT>
__device__ __noinline__ float small_share(const void* row, int e, bool chosen) {
  const float x = chosen ? load_logit<DT>(row, e) : -INFINITY, s = small_score(x, warp_max(x)), all = warp_sum(s);
  return all > 0.0f ? __fdividef(s, all) : 0.0f;
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

// A warp routes one token after another, in fp32 as far as that decides: 3.1 us for a token,
// 5.4 for 2048 of 256 experts, where a token's chain of exchanges is what takes time.  More
// tokens than there are warps at once are bound by the instructions (some 850 a token), and most
// of these calls are for route_many.  Values become sortable keys once, and selection works on
// few of them: the k + 1 largest of the lanes' maxima leave a threshold that at least k + 1
// experts reach and seldom many more.  These (32 at most) go to a lane each, in the order of
// their numbers, which counts those in front of it.  Two neighbours of that order that lie too near
// are put in order in 64 bits, by a lane for each listed expert, and so are the last group that stays
// and the first that does not, by the experts that they may count; where these are not all known or
// too many, the whole token is decided in 64 bits.
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
    const float unit = unit_of(softmax, per);
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
          unsure = next_one && !(value_of(low) - value_of(next_one) > 4.0f * near_of(value_of(low), unit));
        }
      } else if (biased || pair) {
        unsure = out && !(value_of(low) - value_of(out) > 4.0f * near_of(value_of(low), unit));
      }
      if (unsure && whole && biased) {
        // the experts that a group may count, up to a lane each, settle it in 64 bits
        const float v = value_of(pair && second ? second : best);
        const uint32_t from = best ? key_of(v <= FLT_MAX ? v - 4.0f * near_of(v, unit) : v) : 0xffffffffu;
        int have = 0, count;
#pragma unroll
        for (int i = 0; i < VPL; ++i) have += key[i] >= from;
        int at = lanes_before(have, count);
        if (count <= 32) {
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (key[i] >= from) sorted[at++] = e0 + i;
          __syncwarp();
          const int e = lane < count ? sorted[lane] : 0;
          const uint32_t groups = softmax ? groups_exactly<DT, true>(d, row, e, count) : groups_exactly<DT, false>(d, row, e, count);
          kept = real && ((groups >> mine) & 1);
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
      if (__any_sync(kAll, judged && !(v - value_of(sorted[rank + 1]) > near_of(v, unit)))) {
        // where the k-th is clear of what stayed below the threshold, the listed experts settle
        // it among themselves
        const float kth = value_of(sorted[min(d.k, count) - 1]);
        if (few && (least == 1u || kth - value_of(least) > near_of(kth, unit)))
          rank = softmax ? rank_exactly<DT, true>(d, row, me.y, count) : rank_exactly<DT, false>(d, row, me.y, count);
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
      const float all = warp_sum(s);
      s = softmax || all >= 0x1p-30f ? __fdividef(s, all) : small_share<DT>(row, me.y, chosen);
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
  const int64_t ids = 4 * ((d->T - 1) * d->ids_ld + d->k), w = 4 * ((d->T - 1) * d->w_ld + d->k);
  const int64_t logits = static_cast<int64_t>(unit + 1) * ((d->T - 1) * d->logits_ld + d->E);
  MOE_CHECK_ARG(!memory_overlaps(d->topk_ids, ids, d->topk_w, w));
  for (const auto& [out, bytes] : {std::pair<const void*, int64_t>(d->topk_ids, ids), std::pair<const void*, int64_t>(d->topk_w, w)})
    MOE_CHECK_ARG(!memory_overlaps(out, bytes, d->logits, logits) && !memory_overlaps(out, bytes, d->bias, 4ll * d->E) &&
                  !memory_overlaps(out, bytes, d->n_tokens, 4));
  if (int rc = check_device()) return rc;
  int group_lanes = 1;
  while (2 * group_lanes * d->n_group <= 32) group_lanes *= 2;
  if (is_for_route_many(*d)) return route_many(*d, group_lanes, as_stream(stream));
  RouteArgs a{*d, 0, 0, 0, group_lanes};
  if (d->dtype == MOE_DTYPE_F32) return pick_route<MOE_DTYPE_F32>(a, as_stream(stream));
  return d->dtype == MOE_DTYPE_F16 ? pick_route<MOE_DTYPE_F16>(a, as_stream(stream)) : pick_route<MOE_DTYPE_BF16>(a, as_stream(stream));
}
