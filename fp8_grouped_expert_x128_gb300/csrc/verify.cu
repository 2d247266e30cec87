// Verification of drafted tokens against the target's probabilities, and the token
// behind the ones that are taken (moe_verify_drafts).
//
// A cluster of CTAs serves a sequence.  The tests touch two values a draft; what
// takes time is the one row of the target's distribution (and of the draft's, where
// a draft is turned down) that the next token is drawn from.  It is read once: every
// warp sums a run of the vocabulary, the cluster exchanges the warps' sums, and the
// warp whose run holds the border reads its run again, from the L2.
//
// Exactness: a token's borders may lie 1e-9 of the total apart, so sums are those of
// 64-bit arithmetic.  GB300 has few 64-bit units, so a lane sums in pairs of fp32
// (D. E. Knuth's two-sum, TAOCP vol. 2, 4.2.2: sum and rounding error of two numbers
// as two numbers), and only its totals are taken to fp64.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 8;
constexpr uint32_t kAll = 0xffffffffu;

struct VerifyArgs {
  moe_verify_desc d;
};

template <int DT>
__device__ __forceinline__ float prob_at(const void* row, int64_t j) {
  if constexpr (DT == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(row) + j);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(row) + j);
  return DT == MOE_DTYPE_F16 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b);
}

struct Pair {
  float hi = 0.0f, lo = 0.0f;
  // adds s + e, e small beside s
  __device__ __forceinline__ void add(float s, float e) {
    const float t = hi + s, u = t - hi;
    lo += ((hi - (t - u)) + (s - u)) + e;
    hi = t;
  }
};

// w of an entry as a sum of two fp32 numbers: p - q exactly, 0 where that is not a
// positive finite number.
__device__ __forceinline__ void weight_of(float p, float q, float& s, float& e) {
  s = p - q;
  const float u = s - p;
  e = (p - (s - u)) - (q + u);
  if (!(s > 0.0f && s <= FLT_MAX)) s = e = 0.0f;
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

// The distribution that the next token is drawn from.
template <int DT>
struct Weights {
  const void* p;
  const void* q;     // or NULL
  int64_t without;   // an entry that counts as 0, or -1
  __device__ __forceinline__ void at(int64_t j, float& s, float& e) const {
    weight_of(prob_at<DT>(p, j), q ? prob_at<DT>(q, j) : 0.0f, s, e);
    if (j == without) s = e = 0.0f;
  }
};

template <int DT>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ double sums[2][kVerifyWarps];
  const moe_verify_desc& d = a.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y, ctas = gridDim.x, rank = blockIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();

  const int64_t r0 = d.cu_new[b], r1 = d.cu_new[b + 1];
  const int64_t n = d.n_draft ? d.n_draft[b] : r1 - r0 - 1;
  const int32_t len = d.kv_len ? d.kv_len[b] : 0;
  const bool none = r1 == r0 && r0 >= 0 && r1 <= d.T;
  const bool bad = !none && (r0 < 0 || r1 < r0 || r1 > d.T || n < 0 || n >= r1 - r0), wide = !none && !bad && n >= d.max_out;
  if (none || bad || wide) {           // the same for all threads of the cluster
    if (rank == 0) {
      for (int i = threadIdx.x; i < d.max_out; i += kVerifyThreads) d.out_tokens[b * d.out_ld + i] = -1;
      if (threadIdx.x == 0) {
        d.accepted[b] = 0;
        if (d.kv_keep) d.kv_keep[b] = len;
        if (!none) set_err(d.err, bad ? MOE_DEV_BAD_INDEX : MOE_DEV_OVERFLOW);
      }
    }
    return;
  }
  constexpr int kSize = DT == MOE_DTYPE_F32 ? 4 : 2;
  const int64_t s0 = r1 - 1 - n;       // the last token that stands
  auto p_row = [&](int64_t r) { return static_cast<const char*>(d.probs) + r * d.p_ld * kSize; };
  auto q_row = [&](int64_t r) { return static_cast<const char*>(d.draft_probs) + r * d.q_ld * kSize; };
  // every warp tests all drafts, 32 at a time, up to the first that is not taken
  int taken = 0;
  for (; taken < n; taken += 32) {
    bool ok = true;
    if (taken + lane < n) {
      const int64_t r = s0 + taken + lane;
      const int32_t t = d.tokens[r + 1];
      ok = t >= 0 && t < d.vocab;
      if (ok) {
        const double p = prob_at<DT>(p_row(r), t), q = d.draft_probs ? prob_at<DT>(q_row(r), t) : 1.0;
        const float u = d.u_accept[r];
        ok = (u > 0.0f ? static_cast<double>(u) : 0.0) * q < p;
      }
    }
    const uint32_t no = __ballot_sync(kAll, !ok);
    if (no) {
      taken += __ffs(no) - 1;
      break;
    }
  }
  taken = min(taken, static_cast<int>(n));
  const bool refused = taken < n;
  const int64_t row = s0 + taken;
  const int32_t wrong = refused ? d.tokens[row + 1] : -1;
  if (rank == 0) {
    for (int i = threadIdx.x; i < d.max_out; i += kVerifyThreads)
      if (i != taken) d.out_tokens[b * d.out_ld + i] = i < taken ? d.tokens[s0 + 1 + i] : -1;
    if (threadIdx.x == 0) {
      d.accepted[b] = taken;
      if (d.kv_keep) d.kv_keep[b] = len - static_cast<int32_t>(n - taken);
      if (wrong < 0 ? refused : wrong >= d.vocab) set_err(d.err, MOE_DEV_BAD_INDEX);
    }
  }

  // this warp's run of the vocabulary
  const int64_t V = d.vocab, warps = static_cast<int64_t>(ctas) * kVerifyWarps;
  const int64_t len_run = (V + warps - 1) / warps, me = static_cast<int64_t>(rank) * kVerifyWarps + warp;
  const int64_t v0 = min(me * len_run, V), v1 = min(v0 + len_run, V);
  Weights<DT> w{p_row(row), nullptr, -1};
  if (refused) {
    if (d.draft_probs) w.q = q_row(row);
    else w.without = wrong;
  }
  double total = 0.0, before = 0.0, run = 0.0;
  int owner = -1, last = -1;
  for (int pass = 0; pass < 2; ++pass) {
    Pair acc;
    for (int64_t j = v0 + lane; j < v1; j += 32) {
      float s, e;
      w.at(j, s, e);
      acc.add(s, e);
    }
    double sum = static_cast<double>(acc.hi) + static_cast<double>(acc.lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0) sums[pass][warp] = sum;
    cluster_sync_all();
    // every warp: all warps' sums, in the vocabulary's order
    total = before = 0.0;
    owner = last = -1;
    const double u = d.u_sample[b] > 0.0f ? static_cast<double>(d.u_sample[b]) : 0.0;
    auto sum_of = [&](int i) {
      return ld_cluster_f64(cluster_map_shared(smem_u32(&sums[pass][i % kVerifyWarps]), i / kVerifyWarps));
    };
    for (int i = 0; i < warps; ++i) total += sum_of(i);
    const double target = u * total;
    double at = 0.0;
    for (int i = 0; i < warps; ++i) {
      const double x = sum_of(i);
      if (owner < 0 && at + x > target) {
        owner = i;
        before = at;
        run = target;
      }
      if (x > 0.0) last = i;
      at += x;
    }
    if (total > 0.0 || !refused) break;
    w.q = nullptr;                     // nothing is left of the target's distribution: all of it
    w.without = -1;
  }
  const bool beyond = owner < 0;       // u of 1 or more
  if ((beyond ? last : owner) == me) {
    // the first entry of the run whose sum passes the target, or the last that counts
    int64_t found = -1, counts = -1;
    for (int64_t j0 = v0; j0 < v1 && found < 0; j0 += 32) {
      const int64_t j = j0 + lane;
      float s = 0.0f, e = 0.0f;
      if (j < v1) w.at(j, s, e);
      double x = static_cast<double>(s) + static_cast<double>(e);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(kAll, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t some = __ballot_sync(kAll, s > 0.0f);
      const uint32_t over = __ballot_sync(kAll, !beyond && s > 0.0f && before + x > run);
      if (over) found = j0 + __ffs(over) - 1;
      if (some) counts = j0 + 31 - __clz(some);
      before += __shfl_sync(kAll, x, 31);
    }
    if (lane == 0) d.out_tokens[b * d.out_ld + taken] = static_cast<int32_t>(found >= 0 ? found : counts);
  } else if (last < 0 && rank == 0 && threadIdx.x == 0) {   // no entry counts
    d.out_tokens[b * d.out_ld + taken] = -1;
    set_err(d.err, MOE_DEV_BAD_INDEX);
  }
  cluster_sync_all();                  // the others may still read this CTA's sums
}

template <int DT>
int launch_verify(const VerifyArgs& a, cudaStream_t st) {
  // as many CTAs a sequence as fill the GPU, up to a portable cluster
  int ctas = kVerifyMaxCluster;
  while (ctas > 1 && static_cast<int64_t>(a.d.batch) * ctas > 4 * num_sms()) ctas /= 2;
  for (int32_t b0 = 0; b0 < a.d.batch; b0 += 65535) {      // a grid's second dimension
    VerifyArgs part = a;
    part.d.batch = std::min(a.d.batch - b0, 65535);
    part.d.cu_new += b0;
    part.d.u_sample += b0;
    part.d.accepted += b0;
    part.d.out_tokens += b0 * a.d.out_ld;
    if (a.d.n_draft) part.d.n_draft += b0;
    if (a.d.kv_len) part.d.kv_len += b0;
    if (a.d.kv_keep) part.d.kv_keep += b0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, part.d.batch);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, verify_kernel<DT>, part) != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_verify_drafts(const moe_verify_desc* d, void* stream) {
  MOE_CHECK_ARG(d != nullptr && d->flags == 0);
  MOE_CHECK_ARG(d->dtype == MOE_DTYPE_BF16 || d->dtype == MOE_DTYPE_F16 || d->dtype == MOE_DTYPE_F32);
  MOE_CHECK_ARG(d->batch >= 0 && d->T >= 0 && d->vocab >= 1 && d->max_out >= 1 && d->max_out <= 1024);
  MOE_CHECK_ARG(d->p_ld >= d->vocab && (d->draft_probs == nullptr || d->q_ld >= d->vocab) && d->out_ld >= d->max_out);
  MOE_CHECK_ARG((d->kv_len == nullptr) == (d->kv_keep == nullptr));
  if (d->vocab > (1 << 24) || d->batch > (1 << 20) || d->T > (1 << 24) || d->p_ld > INT32_MAX || d->q_ld > INT32_MAX ||
      d->out_ld > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (d->batch == 0) return MOE_OK;
  MOE_CHECK_ARG(d->cu_new && d->u_sample && d->accepted && d->out_tokens);
  MOE_CHECK_ARG(d->T == 0 || (d->probs && d->tokens && d->u_accept));
  const uintptr_t unit = d->dtype == MOE_DTYPE_F32 ? 3 : 1;
  MOE_CHECK_ARG((reinterpret_cast<uintptr_t>(d->probs) & unit) == 0 && (reinterpret_cast<uintptr_t>(d->draft_probs) & unit) == 0);
  const void* words[9] = {d->tokens, d->cu_new, d->n_draft, d->u_accept, d->u_sample, d->kv_len, d->accepted, d->out_tokens, d->kv_keep};
  for (const void* p : words) MOE_CHECK_ARG((reinterpret_cast<uintptr_t>(p) & 3) == 0);
  if (int rc = check_device()) return rc;
  const VerifyArgs a{*d};
  if (d->dtype == MOE_DTYPE_F32) return launch_verify<MOE_DTYPE_F32>(a, as_stream(stream));
  return d->dtype == MOE_DTYPE_F16 ? launch_verify<MOE_DTYPE_F16>(a, as_stream(stream))
                                   : launch_verify<MOE_DTYPE_BF16>(a, as_stream(stream));
}
