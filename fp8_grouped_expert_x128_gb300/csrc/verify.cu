// Verification of drafted tokens against the target's probabilities, and the token
// behind the ones that are taken (moe_verify_drafts).
//
// A cluster of CTAs serves a sequence.  The tests touch two values a draft; what
// takes time is the one row of the target's distribution (and of the draft's, where
// a draft is turned down) that the next token is drawn from.  It is read once: every
// warp sums a run of the vocabulary, the cluster exchanges the warps' sums, and the
// warp whose run holds the border looks for it in its run: between two of the marks at
// which its lanes kept their sums so far, and there a 32nd at a time, from the L2.
//
// 256 sequences of 128000 fp32 entries: 39 us, of which the rows take 32 (6.4 TB/s); the
// exchange (some 5) and the search (2 to 3) come after the rows, as all CTAs go through
// their phases in step.  16 sequences 9.4, 64 15.2, 128 22.4: tests, rows, exchange and search add up.
// One sequence: 6 us, a chain of loads that wait on one another.
//
// Exactness: a token's borders may lie 1e-9 of the total apart, so sums are those of
// 64-bit arithmetic.  GB300 has few 64-bit units (a dependent addition takes 61 cycles,
// and a warp's holds up the SM's other warps), so sums are pairs of fp32 (D. E. Knuth's
// two-sum, TAOCP vol. 2, 4.2.2: sum and rounding error of two numbers as two numbers).
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <utility>

#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 16;
constexpr int kAhead = 4;              // 16-byte loads of a row that a lane has under way
constexpr int kRound = 32 * kAhead;    // vectors of a warp's round of loads
constexpr int kMarks = 8;              // places of a warp's run at which the lanes' sums so far are kept
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
  __device__ __forceinline__ void add(const Pair& o) { add(o.hi, o.lo); }
  // lo below half a unit of hi: then pairs compare by hi first
  __device__ __forceinline__ Pair tidy() const {
    const float t = __fadd_rn(hi, lo);
    return {t, __fadd_rn(__fsub_rn(hi, t), lo)};
  }
  __device__ __forceinline__ bool above(const Pair& o) const {
    const Pair a = tidy(), b = o.tidy();
    return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
  }
};

__device__ __forceinline__ Pair plus(Pair a, const Pair& b) {
  a.add(b);
  return a;
}
__device__ __forceinline__ Pair shfl(const Pair& v, int lane) { return {__shfl_sync(kAll, v.hi, lane), __shfl_sync(kAll, v.lo, lane)}; }

// The sum over the lanes up to and with this one, and of those before it.
__device__ __forceinline__ Pair warp_prefix(Pair x, Pair& before) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y{__shfl_up_sync(kAll, x.hi, o), __shfl_up_sync(kAll, x.lo, o)};
    if (lane >= o) x = plus(y, x);
  }
  before = {__shfl_up_sync(kAll, x.hi, 1), __shfl_up_sync(kAll, x.lo, 1)};
  if (lane == 0) before = Pair{};
  return x;
}

__device__ __forceinline__ void st_cluster_pair(uint32_t addr, const Pair& v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.hi), "f"(v.lo) : "memory");
}

// Two sums at a time, in the packed arithmetic of sm_100 and later.
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.0f, -1.0f), a); }
struct Pairs {
  float2 hi = {0.0f, 0.0f}, lo = {0.0f, 0.0f};
  __device__ __forceinline__ void add(float2 s, float2 e) {
    const float2 t = __fadd2_rn(hi, s), u = sub2(t, hi);
    lo = __fadd2_rn(lo, __fadd2_rn(__fadd2_rn(sub2(hi, sub2(t, u)), sub2(s, u)), e));
    hi = t;
  }
  __device__ __forceinline__ void add(float2 s) {
    const float2 t = __fadd2_rn(hi, s), u = sub2(t, hi);
    lo = __fadd2_rn(lo, __fadd2_rn(sub2(hi, sub2(t, u)), sub2(s, u)));
    hi = t;
  }
  __device__ __forceinline__ Pair sum() const { return plus(Pair{hi.x, lo.x}, Pair{hi.y, lo.y}); }
};

// The distribution that the next token is drawn from: weights p, or max(p - q, 0), in
// vectors of 16 bytes that start where p's addresses are multiples of 16.
template <int DT>
struct Weights {
  static constexpr int kVec = DT == MOE_DTYPE_F32 ? 4 : 8, kSize = 16 / kVec;
  const char* p;      // the row, and q's or NULL
  const char* q;
  int vocab;
  int without;        // an entry that counts as 0, or -1
  int shift;          // entries of vector 0 in front of the row
  int whole0, whole1; // vectors that lie in the row whole
  bool q_wide;        // q's vectors lie like p's
  float careful;      // 0: as they come.  Else entries that are not finite are looked for (they show as a
                      // sum that is not), and the others count this many times

  __device__ __forceinline__ void set(const char* p_row, const char* q_row, int v, int wo) {
    p = p_row;
    q = q_row;
    vocab = v;
    without = wo;
    shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / kSize;
    whole0 = shift > 0;
    whole1 = (shift + vocab) / kVec;
    q_wide = ((reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) & 15) == 0;
    careful = 0.0f;
  }
  __device__ __forceinline__ int vectors() const { return (shift + vocab + kVec - 1) / kVec; }
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
  __device__ __forceinline__ uint4 load(const char* row, int k) const {
    return __ldcs(reinterpret_cast<const uint4*>(row - shift * kSize) + k);
  }
  // vector k of a row that does not lie in it whole, or not at multiples of 16 bytes: zeros outside
  __device__ __noinline__ uint4 piece(const char* row, int k) const {
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; i < kVec; ++i) {
      const int j = k * kVec - shift + i;
      if (j < 0 || j >= vocab) continue;
      if constexpr (DT == MOE_DTYPE_F32) w[i] = __ldg(reinterpret_cast<const uint32_t*>(row) + j);
      else w[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(row) + j)) << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // one entry's weight as the sum of two numbers, 0 where that is not positive and finite
  __device__ __forceinline__ Pair weight(float x, float y) const {
    const float d = __fsub_rn(x, y), u = __fsub_rn(d, x), e = __fsub_rn(__fsub_rn(x, __fsub_rn(d, u)), __fadd_rn(y, u));
    return d > 0.0f && d <= FLT_MAX ? Pair{d, e} : Pair{};
  }
  __device__ __forceinline__ Pair entry(int j) const {
    if (j < 0 || j >= vocab || j == without) return Pair{};
    const Pair v = weight(prob_at<DT>(p, j), q ? prob_at<DT>(q, j) : 0.0f);
    const float times = careful > 0.0f ? careful : 1.0f;      // a power of two
    return {v.hi * times, v.lo * times};
  }
  // The sum of vectors from, from + by, .. below to.  q counts as min(q, p): no comparison is
  // left, and what is not finite shows in the sum.  marks: the sums after `every`, 2 every,
  // .. rounds of loads, 32 places apart.
  template <bool kMarked>
  __device__ __forceinline__ Pair sum(int from, int to, int by, Pair* marks = nullptr, int every = 0) const {
    if (careful > 0.0f) return sum_carefully(from, to, by);
    Pairs acc[2];
    auto round = [&](int k) {
      uint4 a[kAhead], b[kAhead];
      const int last = k + (kAhead - 1) * by;
      if (k >= whole0 && last < min(whole1, to) && q_wide) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) a[i] = load(p, k + i * by);
        if (q != nullptr)
#pragma unroll
          for (int i = 0; i < kAhead; ++i) b[i] = load(q, k + i * by);
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int at = k + i * by;
          const bool inside = at >= whole0 && at < whole1;
          a[i] = b[i] = make_uint4(0, 0, 0, 0);
          if (at < to) {
            a[i] = inside ? load(p, at) : piece(p, at);
            if (q != nullptr) b[i] = inside && q_wide ? load(q, at) : piece(q, at);
          }
        }
      }
      if (q != nullptr) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          float x[kVec], y[kVec];
          unpack(a[i], x);
          unpack(b[i], y);
#pragma unroll
          for (int c = 0; c < kVec; c += 2) {
            const float2 m = make_float2(fminf(y[c], x[c]), fminf(y[c + 1], x[c + 1])), v = make_float2(x[c], x[c + 1]);
            const float2 d = sub2(v, m), u = sub2(d, v);
            acc[c / 2 & 1].add(d, sub2(sub2(v, sub2(d, u)), __fadd2_rn(m, u)));
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          float x[kVec];
          unpack(a[i], x);
          const int out = without - ((k + i * by) * kVec - shift);
          if (without >= 0 && out >= 0 && out < kVec) {
#pragma unroll
            for (int c = 0; c < kVec; ++c) x[c] = c == out ? 0.0f : x[c];
          }
#pragma unroll
          for (int c = 0; c < kVec; c += 2) acc[c / 2 & 1].add(make_float2(fmaxf(x[c], 0.0f), fmaxf(x[c + 1], 0.0f)));
        }
      }
    };
    if constexpr (!kMarked) {
      for (int k = from; k < to; k += kAhead * by) round(k);
      return plus(acc[0].sum(), acc[1].sum());
    }
    Pair all;
    int k = from, end = from / 32 * 32;
#pragma unroll 1
    for (int i = 0; i < kMarks; ++i) {
      end = min(end + every * kAhead * by, to);
#pragma unroll 1
      for (; k < end; k += kAhead * by) round(k);
      marks[32 * i] = all = plus(acc[0].sum(), acc[1].sum());
    }
    return all;
  }
  __device__ __noinline__ Pair sum_carefully(int from, int to, int by) const {
    Pair acc;
    for (int k = from; k < to; k += by)
      for (int i = 0; i < kVec; ++i) acc.add(entry(k * kVec - shift + i));
    return acc;
  }
};

// How a warp's lanes share its run of vectors: each a 32nd of it, whose sum the search then has;
// every 32nd vector each; these, with marks.
enum class Way { kParted, kStrided, kMarked };

template <int DT, Way kWay>
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ Pair sums[2][kVerifyWarps * kVerifyMaxCluster];      // of all warps of the cluster
  __shared__ Pair marks[kWay == Way::kMarked ? kVerifyWarps : 1][kMarks][32];
  const moe_verify_desc& d = a.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y, ctas = gridDim.x, rank = blockIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();

  const int64_t r0 = d.cu_new[b], r1 = d.cu_new[b + 1];
  const int64_t n = d.n_draft ? d.n_draft[b] : r1 - r0 - 1;
  const int32_t len = d.kv_len ? __ldcg(d.kv_len + b) : 0;      // may be kv_keep, whose line others write to
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
  cluster_arrive_relaxed();            // this CTA runs: the others may write to its shared memory
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
  w.set(p_row(row), refused && d.draft_probs ? q_row(row) : nullptr, static_cast<int>(d.vocab), refused && !d.draft_probs ? wrong : -1);
  const int warps = ctas * kVerifyWarps, me = rank * kVerifyWarps + warp;
  const int run = ((w.vectors() + warps - 1) / warps + 31) / 32 * 32;
  int k0 = min(me * run, w.vectors()), k1 = min(k0 + run, w.vectors());
  const int every = (run + kRound * kMarks - 1) / (kRound * kMarks);
  const float u = u_sample > 0.0f ? u_sample : 0.0f;
  const int per = (warps + 31) / 32;            // warps' sums of a lane, at most 4
  constexpr bool kMarked = kWay == Way::kMarked, kParted = kWay == Way::kParted;
  const int f0 = kParted ? min(k0 + lane * (run / 32), k1) : k0 + lane, t0 = kParted ? min(f0 + run / 32, k1) : k1;
  Pair before, target, own;
  int owner = -1;
  bool any = false, beyond = false;
  for (int pass = 0; pass < 6; ++pass) {      // at most: the residual careful and empty, p careful and too large
    own = w.template sum<kMarked>(f0, t0, kParted ? 1 : 32, &marks[kMarked ? warp : 0][0][lane], every);
    Pair sum = own;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum.add(Pair{__shfl_xor_sync(kAll, sum.hi, o), __shfl_xor_sync(kAll, sum.lo, o)});
    // to every CTA of the cluster
    if (pass == 0) cluster_wait();
    if (lane < ctas) st_cluster_pair(cluster_map_shared(smem_u32(&sums[pass & 1][me]), lane), sum);
    __syncwarp();
    cluster_sync_all();
    // every warp: all warps' sums, in the vocabulary's order
    Pair x[4], mine;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = lane * per + i;
      if (i < per && at < warps) x[i] = sums[pass & 1][at];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) mine.add(x[i]);
    Pair at, upto = warp_prefix(mine, at);
    const Pair total = shfl(upto, 31);
    // Infinities among the entries: without them.  Sums of finite ones that are past fp32, or so small
    // that a random number's part of them has bits below fp32's last: of their multiples.
    if (!(total.hi >= 0x1p-90f && total.hi <= FLT_MAX) && total.hi != 0.0f && (w.careful == 0.0f || w.careful == 1.0f)) {
      const bool small = total.hi > 0.0f && total.hi < 1.0f;
      w.careful = small ? 0x1p64f : w.careful == 0.0f ? 1.0f : 0x1p-30f;      // (2^24 entries below 2^128)
      continue;
    }
    any = total.hi > 0.0f;
    if (!any && refused && (w.q != nullptr || w.without >= 0)) {
      w.set(p_row(row), nullptr, static_cast<int>(d.vocab), -1);    // nothing is left of the target's distribution: all of it
      continue;
    }
    // (no sum passes what a u of 1 or more asks for, whatever rounding makes of sums added up in
    // another order)
    target.hi = u < 1.0f ? __fmul_rn(u, total.hi) : INFINITY;
    target.lo = __fmaf_rn(u, total.lo, __fmaf_rn(u, total.hi, -target.hi));
    // the first warp with weight whose sums pass the target, or the last that has some
    int first = -1, last = -1;
    Pair from;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < per) {
        const Pair next = i + 1 == per ? upto : plus(at, x[i]);
        if (first < 0 && x[i].hi > 0.0f && next.above(target)) {
          first = lane * per + i;
          from = at;
        }
        if (x[i].hi > 0.0f) last = lane * per + i;
        at = next;
      }
    const uint32_t over = __ballot_sync(kAll, first >= 0), some = __ballot_sync(kAll, last >= 0);
    if (over) {
      owner = __shfl_sync(kAll, first, __ffs(over) - 1);
      before = shfl(from, __ffs(over) - 1);
    } else if (some) {
      owner = __shfl_sync(kAll, last, 31 - __clz(some));
      beyond = true;                              // u of 1 or more
    }
    break;
  }
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
  if (any && owner == me) {
    if (kMarked && w.careful == 0.0f && !beyond) {
      // the part of the run between two marks, four lanes a mark.  (Not for its last entry with
      // weight: a weight that is small beside the run's does not show in the sums up to the marks.)
      __syncwarp();
      const int i = lane / 4;
      Pair upto;
#pragma unroll
      for (int c = 0; c < 8; ++c) upto.add(marks[warp][i][lane % 4 * 8 + c]);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) upto.add(Pair{__shfl_xor_sync(kAll, upto.hi, o), __shfl_xor_sync(kAll, upto.lo, o)});
      Pair ahead{__shfl_up_sync(kAll, upto.hi, 4), __shfl_up_sync(kAll, upto.lo, 4)};
      if (i == 0) ahead = Pair{};
      const uint32_t over = __ballot_sync(kAll, plus(before, upto).above(target)), some = __ballot_sync(kAll, upto.above(ahead));
      const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
      beyond = over == 0;
      before.add(shfl(ahead, at));
      k0 = min(k0 + at / 4 * every * kRound, k1);
      k1 = min(k0 + every * kRound, k1);
    }
    // the entry in it, a 32nd at a time and then an entry a lane
    auto narrow = [&](int f, int t, const Pair& x) {
      Pair ahead;
      const Pair upto = warp_prefix(x, ahead);
      const uint32_t over = __ballot_sync(kAll, !beyond && x.hi > 0.0f && plus(before, upto).above(target));
      const uint32_t some = __ballot_sync(kAll, x.hi > 0.0f);
      // rounding may leave the border just behind the run: then its last entry
      const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
      beyond |= over == 0;
      before.add(shfl(ahead, at));
      k0 = __shfl_sync(kAll, f, at);
      k1 = __shfl_sync(kAll, t, at);
    };
    if (kParted) narrow(f0, t0, own);
    while ((k1 - k0) * W::kVec > 32) {
      const int piece = (k1 - k0 + 31) / 32, f = min(k0 + lane * piece, k1), t = min(f + piece, k1);
      narrow(f, t, w.template sum<false>(f, t, 1));
    }
    const int j = k0 * W::kVec - w.shift + lane;
    Pair x, ahead;
    if (lane < (k1 - k0) * W::kVec) x = w.entry(j);
    const bool some_of_it = x.hi > 0.0f;
    const Pair upto = warp_prefix(x, ahead);
    const uint32_t over = __ballot_sync(kAll, !beyond && some_of_it && plus(before, upto).above(target)), some = __ballot_sync(kAll, some_of_it);
    if (lane == (over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0)) out[taken] = j;
  }
}

template <int DT, Way kWay>
int launch_verify(const VerifyArgs& a, int ctas, cudaStream_t st) {
  if (ctas > 8) {
    static std::atomic<uint64_t> allowed{0};      // a bit for each GPU that has been told
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (!((allowed.load() >> (dev & 63)) & 1)) {
      MOE_CUDA_TRY(cudaFuncSetAttribute(verify_kernel<DT, kWay>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
      allowed.fetch_or(1ull << (dev & 63));
    }
  }
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
    if (cudaLaunchKernelEx(&cfg, verify_kernel<DT, kWay>, part) != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

template <int DT>
int pick_verify(const VerifyArgs& a, cudaStream_t st) {
  // As many CTAs a sequence as run at once (4 on an SM: 256 sequences of 128000 entries take 39 us,
  // as more, in two goes, 41), but no more than have 32 vectors a warp.  Sixteen to a cluster only
  // where these find room at once (7 clusters).
  const int64_t vectors = a.d.vocab / Weights<DT>::kVec + 2, B = a.d.batch;
  int ctas = 16 * B <= 112 ? 16 : 8;
  while (ctas > 1 && (B * ctas > 4 * num_sms() || (ctas / 2) * kVerifyWarps * 32 >= vectors)) ctas /= 2;
  // Parts where a round of loads takes them whole (37 sequences of 50021 bf16 entries 7.2 -> 6.1 us;
  // of two rounds, one sequence of 128000 in fp32, they take 6.2 and strides 6.05), marks from three
  // rounds on (16 sequences of these 11.1 -> 9.4 us).
  const int64_t rounds = (vectors - 1) / (kRound * kVerifyWarps * ctas);
  if (rounds == 0) return launch_verify<DT, Way::kParted>(a, ctas, st);
  return rounds < 2 ? launch_verify<DT, Way::kStrided>(a, ctas, st) : launch_verify<DT, Way::kMarked>(a, ctas, st);
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
  const int64_t t4 = 4 * d->T, b4 = 4ll * d->batch, size = static_cast<int64_t>(unit) + 1;
  const std::pair<const void*, int64_t> in[8] = {{d->probs, d->T ? size * ((d->T - 1) * d->p_ld + d->vocab) : 0},
                                                 {d->draft_probs, d->T ? size * ((d->T - 1) * d->q_ld + d->vocab) : 0},
                                                 {d->tokens, t4}, {d->cu_new, b4 + 4}, {d->n_draft, b4}, {d->u_accept, t4}, {d->u_sample, b4},
                                                 {d->kv_len, b4}};
  const std::pair<const void*, int64_t> out[3] = {{d->accepted, b4}, {d->out_tokens, 4 * ((d->batch - 1) * d->out_ld + d->max_out)}, {d->kv_keep, b4}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& [p, bytes] : in)
      MOE_CHECK_ARG(!memory_overlaps(out[i].first, out[i].second, p, bytes) || (i == 2 && p == d->kv_len && d->kv_keep == d->kv_len));
    for (int j = 0; j < i; ++j) MOE_CHECK_ARG(!memory_overlaps(out[i].first, out[i].second, out[j].first, out[j].second));
  }
  if (int rc = check_device()) return rc;
  const VerifyArgs a{*d};
  if (d->dtype == MOE_DTYPE_F32) return pick_verify<MOE_DTYPE_F32>(a, as_stream(stream));
  return d->dtype == MOE_DTYPE_F16 ? pick_verify<MOE_DTYPE_F16>(a, as_stream(stream))
                                   : pick_verify<MOE_DTYPE_BF16>(a, as_stream(stream));
}
