// Attention of a step's queries over the paged 8-bit key/value cache.
//
// One warp per (token, query head): the lanes split the head's dimensions, a
// score is a warp sum, and the softmax runs online (running maximum and sum).
#include "kv_attention.cuh"

namespace moe {
namespace {

// cap * tanh(x / cap) in fp32: tanh(y) = 1 - 2 / (exp(2y) + 1).
__device__ __forceinline__ float capped(float x, float cap) {
  const float e = exp2f(2.0f * kLog2e * x / cap);
  return cap * (1.0f - 2.0f / (e + 1.0f));
}

template <bool F16, int D>
__global__ void __launch_bounds__(128) kv_attention_kernel(const __grid_constant__ moe_kv_attention_desc d) {
  const moe_kv_cache& kc = d.cache;
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * 4ll + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / d.q_heads), hq = static_cast<int>(w % d.q_heads);
  if (t >= d.T) return;
  const int b = warp_find(kc.batch, t, [&](int i) { return __ldg(kc.cu_new + i); });
  const int c0 = __ldg(kc.cu_new + b), c1 = __ldg(kc.cu_new + b + 1), len = __ldg(kc.kv_len + b);
  if (t < c0 || t >= c1) return;
  if ((c1 - c0) * (d.q_heads / kc.kv_heads) <= kDecodeRows) return;
  const int P = kc.page_size, h = hq / (d.q_heads / kc.kv_heads);
  if (c0 < 0 || c1 > d.T || len < c1 - c0) {
    if (lane == 0) set_err(d.err, MOE_DEV_BAD_INDEX);
    return;
  }
  if ((len - 1) / P >= kc.max_pages || (d.max_q && c1 - c0 > d.max_q)) {
    if (lane == 0) set_err(d.err, MOE_DEV_OVERFLOW);
    return;
  }
  const int pos = len - (c1 - t);
  const int hi = (d.flags & MOE_KV_FULL) ? len : pos + 1;
  const int lo = d.window > 0 ? max(0, pos - d.window + 1) : 0;
  float q[E], o[E];
  const uint16_t* qp = static_cast<const uint16_t*>(d.q) + t * d.q_token_ld + hq * d.q_head_ld + lane * E;
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float2 p = pair_to_float<F16>(*reinterpret_cast<const uint32_t*>(qp + i));
    q[i] = p.x; q[i + 1] = p.y;
    o[i] = o[i + 1] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = lo; j < hi; ++j) {
    const int page = __ldg(kc.page_table + b * kc.table_ld + j / P);
    if (page < 0 || page >= kc.pages) {
      if (lane == 0) set_err(d.err, MOE_DEV_BAD_INDEX);
      return;
    }
    const uint8_t* kp = kc.k + page * kc.k_page_ld + h * kc.k_head_ld + j % P * kc.k_slot_ld + lane * E;
    const uint8_t* vp = kc.v + page * kc.v_page_ld + h * kc.v_head_ld + j % P * kc.v_slot_ld + lane * E;
    const float ks = __ldg(kc.k_scale + static_cast<int64_t>(page) * kc.kv_heads + h);
    const float vs = __ldg(kc.v_scale + static_cast<int64_t>(page) * kc.kv_heads + h);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const uint32_t p = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kp + i));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
      s = fmaf(q[i], f.x, fmaf(q[i + 1], f.y, s));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= d.sm_scale * ks;
    if (d.softcap > 0.0f) s = capped(s, d.softcap);
    const float mn = fmaxf(m, s);
    const float keep = m == -INFINITY ? 0.0f : exp2f((m - mn) * kLog2e);
    const float p = exp2f((s - mn) * kLog2e);
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const uint32_t c = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vp + i));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c));
      o[i] = o[i] * keep + p * vs * f.x;
      o[i + 1] = o[i + 1] * keep + p * vs * f.y;
    }
    m = mn;
  }
  uint16_t* op = static_cast<uint16_t*>(d.out) + t * d.o_token_ld + hq * d.o_head_ld + lane * E;
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
  for (int i = 0; i < E; i += 2)
    *reinterpret_cast<uint32_t*>(op + i) = pair_from_float<F16>(o[i] * inv, o[i + 1] * inv);
  if (d.lse && lane == 0) d.lse[static_cast<int64_t>(t) * d.q_heads + hq] = l > 0.0f || l != l ? m + logf(l) : -INFINITY;
}

int check_attention(const moe_kv_attention_desc* d) {
  MOE_CHECK_ARG(d != nullptr);
  if (int rc = check_kv_cache(d->cache, d->T)) return rc;
  MOE_CHECK_ARG((d->flags & ~MOE_KV_FULL) == 0);
  MOE_CHECK_ARG(d->q_heads >= 1 && d->q_heads % d->cache.kv_heads == 0);
  MOE_CHECK_ARG(d->max_q >= 0 && d->window >= 0 && !(d->window > 0 && (d->flags & MOE_KV_FULL)));
  MOE_CHECK_ARG(isfinite(d->sm_scale) && isfinite(d->softcap) && d->softcap >= 0.0f);
  MOE_CHECK_ARG(kv_strides_ok(d->q_token_ld, d->q_head_ld, d->o_token_ld, 8) && kv_strides_ok(d->o_head_ld, 0, 0, 8));
  if (d->q_heads > 65536 || d->T * d->q_heads > (1ll << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_kv_attention_workspace_size(const moe_kv_attention_desc* d) {
  return check_attention(d) == MOE_OK ? kv_decode_workspace() : 0;
}

extern "C" int moe_kv_attention(const moe_kv_attention_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_attention(d)) return rc;
  if (d->T == 0 || d->cache.batch == 0) return MOE_OK;
  MOE_CHECK_ARG(d->q && d->out && aligned16(d->q) && aligned16(d->out));
  MOE_CHECK_ARG(workspace != nullptr && (reinterpret_cast<uintptr_t>(workspace) & 255) == 0);
  MOE_CHECK_ARG(workspace_bytes >= moe_kv_attention_workspace_size(d));
  if (int rc = check_device()) return rc;
  AttnArgs a{};
  a.d = *d;
  a.G = d->q_heads / d->cache.kv_heads;
  a.counters = static_cast<int32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(a.counters + kDecodeCounters);
  const int64_t max_rows = (d->max_q ? static_cast<int64_t>(d->max_q) : d->T) * a.G;
  if (int rc = kv_decode_launch(a, max_rows, as_stream(stream))) return rc;
  if (max_rows <= kDecodeRows) return MOE_OK;
  const dim3 grid(static_cast<unsigned>((d->T * d->q_heads + 3) / 4));
  cudaStream_t st = as_stream(stream);
  const bool f16 = d->cache.dtype == MOE_DTYPE_F16;
  if (d->cache.dim == 64)
    return f16 ? launch_pdl(kv_attention_kernel<true, 64>, grid, dim3(128), 0, st, *d)
               : launch_pdl(kv_attention_kernel<false, 64>, grid, dim3(128), 0, st, *d);
  return f16 ? launch_pdl(kv_attention_kernel<true, 128>, grid, dim3(128), 0, st, *d)
             : launch_pdl(kv_attention_kernel<false, 128>, grid, dim3(128), 0, st, *d);
}
