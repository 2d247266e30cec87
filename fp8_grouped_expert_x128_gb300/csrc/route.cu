// Routing to experts: softmax or sigmoid scores, a bias for balance, groups,
// top-k, renormalised weights (moe_route).
#include <cfloat>
#include <cmath>

#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kRouteWarps = 4;      // tokens of a CTA, a warp each
constexpr uint32_t kAll = 0xffffffffu;

struct RouteArgs {
  moe_route_desc d;
};

// A logit as fp32: NaN and -inf (an expert that is not open) become -inf, +inf the
// largest fp32.
__device__ __forceinline__ float as_logit(float z) { return z > -INFINITY ? fminf(z, FLT_MAX) : -INFINITY; }

template <int DT>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  if constexpr (DT == MOE_DTYPE_F32) return as_logit(__ldg(static_cast<const float*>(row) + e));
  const uint16_t b = __ldg(static_cast<const uint16_t*>(row) + e);
  return as_logit(DT == MOE_DTYPE_F16 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b));
}

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The largest (value, lowest number) of the lanes' candidates; number < 0: none.
__device__ __forceinline__ void warp_best(double& v, int& n) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(kAll, v, o);
    const int on = __shfl_xor_sync(kAll, n, o);
    if (on >= 0 && (n < 0 || ov > v || (ov == v && on < n))) {
      v = ov;
      n = on;
    }
  }
}

// One token in 64-bit arithmetic by one warp.  value: E doubles of shared memory.
// Lane j < k gets the number of the j-th expert, -1 where there is none.
template <int DT>
__device__ __noinline__ int route_exact(const moe_route_desc& d, const void* row, double* value) {
  const int lane = threadIdx.x & 31;
  const bool softmax = d.flags & MOE_ROUTE_SOFTMAX, pair = d.flags & MOE_ROUTE_GROUP_PAIR;
  double top = -INFINITY, sum = 1.0;
  if (softmax) {
    for (int e = lane; e < d.E; e += 32) top = fmax(top, static_cast<double>(load_logit<DT>(row, e)));
    top = warp_max(top);
    sum = 0.0;
    for (int e = lane; e < d.E; e += 32) {
      const float z = load_logit<DT>(row, e);
      if (z > -INFINITY) sum += exp(z - top);
    }
    sum = warp_sum(sum);
  }
  auto score = [&](float z) { return softmax ? exp(z - top) / sum : 1.0 / (1.0 + exp(-static_cast<double>(z))); };
  for (int e = lane; e < d.E; e += 32) {
    const float z = load_logit<DT>(row, e);
    double v = z;
    if (d.bias != nullptr) {
      const float b = __ldg(d.bias + e);
      v = (z > -INFINITY && b > -INFINITY) ? score(z) + b : -INFINITY;
    }
    value[e] = v;
  }
  __syncwarp();
  const int size = d.E / d.n_group;
  uint32_t kept = kAll;
  if (d.n_group > 1) {
    // lane g: group g
    double mine = -INFINITY;
    if (lane < d.n_group) {
      double a = -INFINITY, b = -INFINITY;
      for (int i = 0; i < size; ++i) {
        double v = value[lane * size + i];
        if (pair && d.bias == nullptr && v > -INFINITY) v = score(static_cast<float>(v));
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
      mine = (pair && b > -INFINITY) ? a + b : a;
    }
    kept = 0;
    for (int r = 0; r < d.topk_group; ++r) {
      double v = mine;
      int n = (lane < d.n_group && !((kept >> lane) & 1)) ? lane : -1;
      warp_best(v, n);
      if (n >= 0) kept |= 1u << n;
    }
  }
  int found = -1;
  for (int j = 0; j < d.k; ++j) {
    double v = -INFINITY;
    int n = -1;
    for (int e = lane; e < d.E; e += 32) {
      const double x = value[e];
      if (x > -INFINITY && (d.n_group == 1 || ((kept >> (e / size)) & 1)) && (n < 0 || x > v)) {
        v = x;
        n = e;
      }
    }
    warp_best(v, n);
    if (n < 0) break;
    if (lane == j) found = n;
    if (lane == (n & 31)) value[n] = -INFINITY;
    __syncwarp();
  }
  __syncwarp();
  return found;
}

template <int DT>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ double route_smem[];
  const moe_route_desc& d = a.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t >= d.T) return;
  constexpr int kSize = DT == MOE_DTYPE_F32 ? 4 : 2;
  const void* row = static_cast<const char*>(d.logits) + t * d.logits_ld * kSize;
  int id = -1;
  if (d.n_tokens == nullptr || t < *d.n_tokens) id = route_exact<DT>(d, row, route_smem + static_cast<size_t>(warp) * d.E);
  // the weights of the chosen ones, in fp32
  float s = 0.0f;
  if (d.flags & MOE_ROUTE_SOFTMAX) {
    float top = -INFINITY;
    for (int e = lane; e < d.E; e += 32) top = fmaxf(top, load_logit<DT>(row, e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    float sum = 0.0f;
    for (int e = lane; e < d.E; e += 32) {
      const float z = load_logit<DT>(row, e);
      if (z > -INFINITY) sum += expf(z - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (id >= 0) s = expf(load_logit<DT>(row, id) - top) / sum;
  } else if (id >= 0) {
    s = 1.0f / (1.0f + expf(-load_logit<DT>(row, id)));
  }
  if (d.flags & MOE_ROUTE_RENORM) {
    float sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    s = sum > 0.0f ? s / sum : 0.0f;
  }
  if (lane < d.k) {
    d.topk_ids[t * d.ids_ld + lane] = id;
    d.topk_w[t * d.w_ld + lane] = s * d.scale;
  }
}

template <int DT>
int launch_route(const RouteArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(double) * kRouteWarps * a.d.E;
  return launch_pdl(route_kernel<DT>, dim3(static_cast<unsigned>((a.d.T + kRouteWarps - 1) / kRouteWarps)), dim3(32 * kRouteWarps),
                    smem, st, a);
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
  const RouteArgs a{*d};
  if (d->dtype == MOE_DTYPE_F32) return launch_route<MOE_DTYPE_F32>(a, as_stream(stream));
  return d->dtype == MOE_DTYPE_F16 ? launch_route<MOE_DTYPE_F16>(a, as_stream(stream))
                                   : launch_route<MOE_DTYPE_BF16>(a, as_stream(stream));
}
