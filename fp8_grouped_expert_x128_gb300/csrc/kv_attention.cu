// Attention of a step's queries over the paged 8-bit key/value cache: the entry
// point, which checks the descriptor and launches the kernel for sequences with
// few rows (kv_decode.cu), the one for many (kv_prefill.cu), or both.
#include "kv_attention.cuh"

namespace moe {
namespace {

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
  if (check_attention(d) != MOE_OK) return 0;
  const size_t few = kv_decode_workspace(), many = kv_prefill_workspace();
  return kDecodeCounters * sizeof(int32_t) + (few > many ? few : many);
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
  if (d->softcap > 0.0f) a.d.softcap = fminf(fmaxf(d->softcap, kMinCap), kMaxCap);
  a.G = d->q_heads / d->cache.kv_heads;
  a.counters = static_cast<int32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(a.counters + kDecodeCounters);
  const int64_t max_rows = (d->max_q ? static_cast<int64_t>(d->max_q) : d->T) * a.G;
  if (int rc = kv_decode_launch(a, max_rows, as_stream(stream))) return rc;
  if (max_rows <= kDecodeRows) return MOE_OK;
  return kv_prefill_launch(a, as_stream(stream));
}
