// The router's logits: tokens times the gate's rows, fp32 sums (moe_gate).
#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kGateTile = 64, kGateK = 16;

template <bool F16>
__device__ __forceinline__ float one_value(uint16_t b) {
  return F16 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b);
}

// 64 x 64 logits a CTA, 4 x 4 a thread.
template <bool F16>
__global__ void __launch_bounds__(256) gate_kernel(const __grid_constant__ moe_gate_desc d) {
  __shared__ float xs[kGateK][kGateTile + 1], ws[kGateK][kGateTile + 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGateTile;
  const int e0 = blockIdx.y * kGateTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int h0 = 0; h0 < d.H; h0 += kGateK) {
    for (int i = threadIdx.x; i < kGateK * kGateTile; i += 256) {
      const int r = i / kGateK, h = h0 + i % kGateK;
      xs[i % kGateK][r] = (t0 + r < d.T && h < d.H) ? one_value<F16>(static_cast<const uint16_t*>(d.x)[(t0 + r) * d.x_ld + h]) : 0.0f;
      ws[i % kGateK][r] = (e0 + r < d.E && h < d.H) ? one_value<F16>(static_cast<const uint16_t*>(d.w)[(e0 + r) * d.w_ld + h]) : 0.0f;
    }
    __syncthreads();
    float part[4][4] = {};
    for (int k = 0; k < kGateK; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], part[i][j]);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) acc[i][j] += part[i][j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (t0 + ty + 16 * i < d.T && e0 + tx + 16 * j < d.E) d.logits[(t0 + ty + 16 * i) * d.logits_ld + e0 + tx + 16 * j] = acc[i][j];
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_gate(const moe_gate_desc* d, void* stream) {
  MOE_CHECK_ARG(d != nullptr && d->flags == 0);
  MOE_CHECK_ARG(d->dtype == MOE_DTYPE_BF16 || d->dtype == MOE_DTYPE_F16);
  MOE_CHECK_ARG(d->T >= 0 && d->E >= 1 && d->H >= 8 && d->H % 8 == 0);
  MOE_CHECK_ARG(d->x_ld >= d->H && d->w_ld >= d->H && d->x_ld % 8 == 0 && d->w_ld % 8 == 0 && d->logits_ld >= d->E);
  if (d->E > 1024 || d->H > (1 << 20) || d->T > (1 << 24) || d->x_ld > INT32_MAX || d->w_ld > INT32_MAX || d->logits_ld > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (d->T == 0) return MOE_OK;
  MOE_CHECK_ARG(d->x && d->w && d->logits && aligned16(d->x) && aligned16(d->w) && (reinterpret_cast<uintptr_t>(d->logits) & 3) == 0);
  if (int rc = check_device()) return rc;
  const dim3 grid(static_cast<unsigned>((d->T + kGateTile - 1) / kGateTile), (d->E + kGateTile - 1) / kGateTile);
  return d->dtype == MOE_DTYPE_F16 ? launch_pdl(gate_kernel<true>, grid, dim3(256), 0, as_stream(stream), *d)
                                   : launch_pdl(gate_kernel<false>, grid, dim3(256), 0, as_stream(stream), *d);
}
