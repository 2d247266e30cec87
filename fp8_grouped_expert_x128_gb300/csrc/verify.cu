// Verification of drafted tokens against the target's probabilities, and the token
// behind the ones that are taken (moe_verify_drafts).
//
// A cluster of CTAs serves a sequence.  The tests touch two values a draft; what
// takes time is the one row of the target's distribution (and of the draft's, where
// a draft is turned down) that the next token is drawn from.  It is read once: every
// warp sums a run of the vocabulary, the cluster exchanges the warps' sums, and the
// warp whose run holds the border looks for it in its run, a 32nd at a time, from the
// L2.
//
// Exactness: a token's borders may lie 1e-9 of the total apart, so sums are those of
// 64-bit arithmetic.  GB300 has few 64-bit units (a dependent addition takes 61 cycles),
// so a lane sums in pairs of fp32 (D. E. Knuth's two-sum, TAOCP vol. 2, 4.2.2: sum and
// rounding error of two numbers as two numbers), and only warps' totals are taken to fp64.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kAhead = 4;              // 16-byte loads of a row that a lane has under way
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

// A sum and what its rounding lost.
struct Pair {
  float hi = 0.0f, lo = 0.0f;
  // adds s + e, e small beside s
  __device__ __forceinline__ void add(float s, float e) {
    const float t = __fadd_rn(hi, s), u = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(t, u)), __fsub_rn(s, u)), e));
    hi = t;
  }
};

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

// The distribution that the next token is drawn from: weights p, or max(p - q, 0), in
// vectors of 16 bytes that start where p's addresses are multiples of 16.
template <int DT>
struct Weights {
  static constexpr int kVec = DT == MOE_DTYPE_F32 ? 4 : 8, kSize = 16 / kVec;
  const char* p;
  const char* q;      // or NULL
  int64_t vocab;
  int64_t without;    // an entry that counts as 0, or -1
  int shift;          // entries of vector 0 in front of the row
  bool q_wide;        // q's vectors lie like p's
  bool careful;       // infinities are looked for (else they show as a sum that is not finite)

  __device__ __forceinline__ void set(const char* p_row, const char* q_row, int64_t v, int64_t wo) {
    p = p_row;
    q = q_row;
    vocab = v;
    without = wo;
    shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / kSize;
    q_wide = ((reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) & 15) == 0;
    careful = false;
  }
  __device__ __forceinline__ int64_t vectors() const { return (shift + vocab + kVec - 1) / kVec; }
  // vectors [k, k + n) inside the row
  __device__ __forceinline__ bool inside(int64_t k, int64_t n) const {
    return k * kVec >= shift && (k + n) * kVec <= shift + vocab;
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[kVec]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE_DTYPE_F32) {
        f[i] = __uint_as_float(w[i]);
      } else {
        const float2 v = pair_to_float<DT == MOE_DTYPE_F16>(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  }
  static __device__ __forceinline__ uint4 load(const char* row, int64_t k, int shift) {
    return __ldcs(reinterpret_cast<const uint4*>(row - shift * kSize) + k);
  }
  // p - q as the sum of two numbers, 0 where that is not positive (or NaN)
  __device__ __forceinline__ void weight(float x, float y, float& s, float& e) const {
    const float d = __fsub_rn(x, y), u = __fsub_rn(d, x);
    e = __fsub_rn(__fsub_rn(x, __fsub_rn(d, u)), __fadd_rn(y, u));
    e = d > 0.0f ? e : 0.0f;
    s = fmaxf(d, 0.0f);
    if (careful && !(s <= FLT_MAX)) s = e = 0.0f;
  }
  __device__ __forceinline__ void weight(float x, float& s) const {
    s = fmaxf(x, 0.0f);
    if (careful && !(s <= FLT_MAX)) s = 0.0f;
  }
  // vector k's weights, whatever of it is in the row
  __device__ __forceinline__ void get(int64_t k, float (&s)[kVec], float (&e)[kVec]) const {
    float x[kVec], y[kVec];
    const int64_t j0 = k * kVec - shift;
    if (inside(k, 1)) {
      unpack(load(p, k, shift), x);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[i] = j0 + i >= 0 && j0 + i < vocab ? prob_at<DT>(p, j0 + i) : 0.0f;
    }
    if (q != nullptr && inside(k, 1) && q_wide) {
      unpack(load(q, k, shift), y);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) y[i] = q != nullptr && j0 + i >= 0 && j0 + i < vocab ? prob_at<DT>(q, j0 + i) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      weight(x[i], y[i], s[i], e[i]);
      if (j0 + i == without) s[i] = e[i] = 0.0f;
    }
  }
  // the sum of vectors from, from + by, .. below to
  __device__ __forceinline__ double sum(int64_t from, int64_t to, int by) const {
    Pair acc[4];
    const bool wide = q == nullptr || q_wide;
    int64_t k = from;
    for (; k + (kAhead - 1) * by < to; k += kAhead * by) {
      const int64_t j0 = k * kVec - shift, j1 = (k + (kAhead - 1) * by + 1) * kVec - shift;
      if (wide && inside(k, (kAhead - 1) * by + 1) && !(without >= j0 && without < j1)) {
        uint4 a[kAhead], b[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) a[i] = load(p, k + i * by, shift);
        if (q != nullptr) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) b[i] = load(q, k + i * by, shift);
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            float x[kVec], y[kVec];
            unpack(a[i], x);
            unpack(b[i], y);
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
              float s, e;
              weight(x[c], y[c], s, e);
              acc[c & 3].add(s, e);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            float x[kVec];
            unpack(a[i], x);
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
              float s;
              weight(x[c], s);
              acc[c & 3].add(s, 0.0f);
            }
          }
        }
      } else {
        for (int i = 0; i < kAhead; ++i) add_one(k + i * by, acc);
      }
    }
    for (; k < to; k += by) add_one(k, acc);
    acc[0].add(acc[1].hi, acc[1].lo);
    acc[2].add(acc[3].hi, acc[3].lo);
    acc[0].add(acc[2].hi, acc[2].lo);
    return static_cast<double>(acc[0].hi) + static_cast<double>(acc[0].lo);
  }

 private:
  __device__ __forceinline__ void add_one(int64_t k, Pair (&acc)[4]) const {
    float s[kVec], e[kVec];
    get(k, s, e);
#pragma unroll
    for (int c = 0; c < kVec; ++c) acc[c & 3].add(s[c], e[c]);
  }
};

__device__ __forceinline__ double warp_prefix(double x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

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
  const float u_sample = d.u_sample[b];
  const bool none = r1 == r0 && r0 >= 0 && r1 <= d.T;
  const bool bad = !none && (r0 < 0 || r1 < r0 || r1 > d.T || n < 0 || n >= r1 - r0), wide = !none && !bad && n >= d.max_out;
  int32_t* out = d.out_tokens + b * d.out_ld;
  if (none || bad || wide) {           // the same for all threads of the cluster
    if (rank == 0) {
      for (int i = threadIdx.x; i < d.max_out; i += kVerifyThreads) out[i] = -1;
      if (threadIdx.x == 0) {
        d.accepted[b] = 0;
        if (d.kv_keep) d.kv_keep[b] = len;
        if (!none) set_err(d.err, bad ? MOE_DEV_BAD_INDEX : MOE_DEV_OVERFLOW);
      }
    }
    return;
  }
  using W = Weights<DT>;
  const int64_t s0 = r1 - 1 - n;       // the last token that stands
  auto p_row = [&](int64_t r) { return static_cast<const char*>(d.probs) + r * d.p_ld * W::kSize; };
  auto q_row = [&](int64_t r) { return static_cast<const char*>(d.draft_probs) + r * d.q_ld * W::kSize; };
  // every warp tests all drafts, 32 at a time, up to the first that is not taken
  int taken = 0;
  for (; taken < n; taken += 32) {
    bool ok = true;
    if (taken + lane < n) {
      const int64_t r = s0 + taken + lane;
      const int32_t t = d.tokens[r + 1];
      const float u = d.u_accept[r];
      ok = t >= 0 && t < d.vocab;
      if (ok) {
        const double p = prob_at<DT>(p_row(r), t), q = d.draft_probs ? prob_at<DT>(q_row(r), t) : 1.0;
        ok = (u > 0.0f ? static_cast<double>(u) : 0.0) * q < p;      // exact: 24 bits by 24
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

  // this warp's run of the vocabulary
  W w;
  w.set(p_row(row), refused && d.draft_probs ? q_row(row) : nullptr, d.vocab, refused && !d.draft_probs ? wrong : -1);
  const int warps = ctas * kVerifyWarps, me = rank * kVerifyWarps + warp;
  const int64_t run = ((w.vectors() + warps - 1) / warps + 31) / 32 * 32;
  int64_t k0 = min(me * run, w.vectors()), k1 = min(k0 + run, w.vectors());
  const double u = u_sample > 0.0f ? static_cast<double>(u_sample) : 0.0;
  const int per = (warps + 31) / 32;            // warps' sums of a lane, at most 4
  double before = 0.0, target = 0.0;
  int owner = -1;
  bool any = false;
  for (int pass = 0; pass < 4; ++pass) {
    double sum = w.sum(k0 + lane, k1, 32);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0) sums[pass & 1][warp] = sum;
    __syncwarp();
    cluster_sync_all();
    // every warp: all warps' sums, in the vocabulary's order
    double x[4], mine = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = lane * per + i;
      x[i] = i < per && at < warps ? ld_cluster_f64(cluster_map_shared(smem_u32(&sums[pass & 1][at % kVerifyWarps]), at / kVerifyWarps)) : 0.0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) mine += x[i];
    const double upto = warp_prefix(mine);
    const double total = __shfl_sync(kAll, upto, 31);
    if (!isfinite(total) && !w.careful) {       // infinities among the entries: without them
      w.careful = true;
      continue;
    }
    any = total > 0.0;
    if (!any && refused && (w.q != nullptr || w.without >= 0)) {
      w.set(p_row(row), nullptr, d.vocab, -1);    // nothing is left of the target's distribution: all of it
      // (its vectors are the same ones)
      continue;
    }
    target = u * total;
    // the first warp whose sums pass the target, or the last that has some
    int first = -1, last = -1;
    double at = upto - mine, from = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) {
        const double next = i + 1 == per ? upto : at + x[i];
        if (first < 0 && next > target) {
          first = lane * per + i;
          from = at;
        }
        if (x[i] > 0.0) last = lane * per + i;
        at = next;
      }
    const uint32_t over = __ballot_sync(kAll, first >= 0), some = __ballot_sync(kAll, last >= 0);
    if (over) {
      owner = __shfl_sync(kAll, first, __ffs(over) - 1);
      before = __shfl_sync(kAll, from, __ffs(over) - 1);
    } else if (some) {
      owner = __shfl_sync(kAll, last, 31 - __clz(some));
      target = INFINITY;
    }
    break;
  }
  __syncwarp();
  cluster_sync_relaxed();                       // the others have read this CTA's sums
  if (rank == 0) {
    for (int i = threadIdx.x; i < d.max_out; i += kVerifyThreads)
      if (i != taken) out[i] = i < taken ? d.tokens[s0 + 1 + i] : -1;
    if (threadIdx.x == 0) {
      d.accepted[b] = taken;
      if (d.kv_keep) d.kv_keep[b] = len - static_cast<int32_t>(n - taken);
      if (!any) out[taken] = -1;
      if (!any || (refused && (wrong < 0 || wrong >= d.vocab))) set_err(d.err, MOE_DEV_BAD_INDEX);
    }
  }
  if (!any || owner != me) return;
  // the vector in the run, a 32nd at a time
  for (;;) {
    const int64_t piece = (k1 - k0 + 31) / 32, f = min(k0 + lane * piece, k1), t = min(f + piece, k1);
    const double x = w.sum(f, t, 1), upto = warp_prefix(x);
    const uint32_t over = __ballot_sync(kAll, x > 0.0 && before + upto > target), some = __ballot_sync(kAll, x > 0.0);
    // rounding may leave the border just behind the run: then its last entry
    const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
    if (!over) target = INFINITY;
    before += __shfl_sync(kAll, upto - x, at);
    k0 = __shfl_sync(kAll, f, at);
    k1 = __shfl_sync(kAll, t, at);
    if (piece <= 1) break;
  }
  if (lane == 0) {
    float s[W::kVec], e[W::kVec];
    w.get(k0, s, e);
    int found = -1, last = 0;
#pragma unroll
    for (int i = 0; i < W::kVec; ++i) {
      before += static_cast<double>(s[i]) + static_cast<double>(e[i]);
      if (s[i] > 0.0f) {
        last = i;
        if (found < 0 && before > target) found = i;
      }
    }
    out[taken] = static_cast<int32_t>(k0 * W::kVec - w.shift + (found >= 0 ? found : last));
  }
}

template <int DT>
int launch_verify(const VerifyArgs& a, cudaStream_t st) {
  // As many CTAs a sequence as fill the GPU (8 on an SM), but no more than have 32 vectors a
  // warp.  Sixteen to a cluster only where these find room at once (7 clusters).
  const int64_t vectors = a.d.vocab / Weights<DT>::kVec + 2, B = a.d.batch;
  int ctas = 16 * B <= 112 ? 16 : 8;
  while (ctas > 1 && (B * ctas > 8 * num_sms() || (ctas / 2) * kVerifyWarps * 32 >= vectors)) ctas /= 2;
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
    if (ctas > 8) MOE_CUDA_TRY(cudaFuncSetAttribute(verify_kernel<DT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
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
