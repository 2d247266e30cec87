// Appending a step's keys and values to the paged 8-bit cache, with the position
// rotation of keys and queries on the way.
//
// Per page, head and K or V: s' = the power-of-two scale of the page's new
// tokens (and of what the page held before), q = e4m3(x / s').  The maximum has
// to be known before the first code is written.  Bound by HBM for prompts, by the
// chain of dependent loads (sequence, page, rows) for single tokens; two kernels:
//
// kv_append_pages_kernel, for prompts: a CTA takes one page and one of K or V,
// keeps the page's rotated rows in registers (fp32, 16 values a thread and row),
// takes the maximum over the CTA and then writes the codes: the inputs are read
// once.  It walks over several heads, the next head's rows loading meanwhile, so
// that the chain is paid once for all of them.
//
// kv_append_tokens_kernel, for few new tokens a page: a CTA takes one page with all
// its heads, K and V; 4 or 8 lanes share a row, and the maximum stays among them.
//
// Measured: 256 single tokens with 32 query and 8 kv heads 5.4 us on the GPU; 32768
// prompt tokens with 64 and 8 heads 210 us, 6.1 TB/s (91% of a copy's rate), of which
// the queries 154 at the copy's rate and the pages 56; ragged chunks of 64-dimension
// heads, f16, token-major pages 44 us by graph replay, 3.7 TB/s (4 KB a head and CTA, a barrier each).
//
// Query rows need no maximum: further CTAs of the tokens kernel's launch rotate them,
// and for prompts a kernel of its own, with the registers that suit it.
#include <float.h>

#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kQHeadsPerCta = 4;   // query heads one thread rotates with the same angles
constexpr int kFewTokens = 4;      // new tokens a sequence, on average, up to which the tokens kernel serves

struct AppendArgs {
  moe_kv_append_desc d;
  int32_t units;        // page units: floor(T / page_size) + 2 * batch
  int32_t head_groups;  // CTAs per unit and kind
  int32_t heads_per;    // kv heads per CTA
  int32_t kv_ctas;      // CTAs before those of the queries (tokens kernel) and the checks
  int32_t q_ctas;       // tokens kernel: of the queries
  int32_t q_groups;     // CTAs per run of query rows
};

// A thread's 16 dimensions of a row: two runs of 8.  Where dimensions (i, i +
// rot / 2) turn together the runs are rot / 2 apart, so that both ends of a pair
// are in one thread; else they are neighbours.
__device__ __forceinline__ void group_runs(int g, int rot, bool interleaved, int& a, int& b) {
  const int rg = rot >> 4;
  if (!interleaved && g < rg) {
    a = 8 * g;
    b = 8 * (g + rg);
  } else {
    a = 16 * g;
    b = 16 * g + 8;
  }
}

__device__ __forceinline__ void load8f(const float* p, float (&f)[8]) {
  const float4 u = __ldg(reinterpret_cast<const float4*>(p)), v = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
  f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
}

__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8],
                                     bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = b * c[i] + a * s[i];
      a = y[2 * i], b = y[2 * i + 1];
      y[2 * i] = a * c[4 + i] - b * s[4 + i];
      y[2 * i + 1] = b * c[4 + i] + a * s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = y[i];
      x[i] = a * c[i] - b * s[i];
      y[i] = b * c[i] + a * s[i];
    }
  }
}

// |x| where x is finite, else 0: what counts toward a page's maximum.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.0f;
}
// max(amax, |x|, |y|): NaN takes no part, infinity does; with an infinite maximum the
// caller takes it again over the finite values.
__device__ __forceinline__ float abs_max(const float (&x)[8], const float (&y)[8], float amax) {
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(fmaxf(amax, fabsf(x[i])), fabsf(y[i]));
  return amax;
}
__device__ __forceinline__ float finite_max(const float (&x)[8], const float (&y)[8], float amax) {
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(fmaxf(amax, finite_abs(x[i])), finite_abs(y[i]));
  return amax;
}

// e4m3(x / s): a product with the exact reciprocal where s is a power of two.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, bool pow2) {
  float q[8];
  if (pow2) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = x[i] * r;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], s);
  }
  return pack_e4m3x8(q);
}

// What is wrong with a sequence that has new tokens, so that it is skipped whole; 0: nothing.
__device__ __forceinline__ int32_t sequence_fault(const moe_kv_append_desc& d, int c0, int c1, int len) {
  if (c0 < 0 || c1 < c0 || c1 > d.T || len < c1 - c0) return MOE_DEV_BAD_INDEX;
  return len > d.cache.max_pages * d.cache.page_size ? MOE_DEV_OVERFLOW : 0;
}

// Offsets that decrease lead the search past sequences, whose CTAs then cannot tell of
// them: the last CTAs look at the offsets alone, a thread for each sequence.  (In the CTAs
// of the units, two more loads each, it took 256 single tokens from 5.2 to 6.1 us; here 5.4.)
template <int TT>
__device__ __forceinline__ void check_offsets(const moe_kv_append_desc& d, int cta) {
  const int b = cta * TT + threadIdx.x;
  if (b >= d.cache.batch) return;
  const int c0 = __ldg(d.cache.cu_new + b);
  if (c0 < 0 || __ldg(d.cache.cu_new + b + 1) < c0) set_err(d.err, MOE_DEV_BAD_INDEX);
}
template <int TT>
int check_ctas(const AppendArgs& a) {
  return (a.d.cache.batch + TT - 1) / TT;
}

template <bool F16, int D, int TT>
__device__ void rotate_queries(const AppendArgs& a, int cta) {
  const moe_kv_append_desc& d = a.d;
  constexpr int kGroups = D / 16;
  constexpr int kRows = TT / kGroups;
  const int t = cta / a.q_groups * kRows + threadIdx.x / kGroups;
  const int t_warp = min(t, static_cast<int>(d.T) - 1);
  const int g = threadIdx.x % kGroups;
  const int h0 = cta % a.q_groups * kQHeadsPerCta;
  const int h1 = min(h0 + kQHeadsPerCta, d.q_heads);
  // the lanes of a warp hold different rows: each searches for its own
  int lo = 0, hi = d.cache.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(d.cache.cu_new + mid) <= t_warp) lo = mid; else hi = mid;
  }
  const int c0 = __ldg(d.cache.cu_new + lo), c1 = __ldg(d.cache.cu_new + lo + 1), len = __ldg(d.cache.kv_len + lo);
  if (t >= d.T || t < c0 || t >= c1 || sequence_fault(d, c0, c1, len)) return;   // the pages' CTAs tell of faults
  const int pos = len - (c1 - t);
  if (d.rot_dim && pos >= d.max_pos) {
    set_err(d.err, MOE_DEV_BAD_INDEX);
    return;
  }
  const bool inter = (d.flags & MOE_KV_INTERLEAVED) != 0;
  const bool turned = g < (d.rot_dim >> 4);
  int ra, rb;
  group_runs(g, d.rot_dim, inter, ra, rb);
  float c[8], s[8];
  if (turned) {
    const float* cs = d.cos_sin + static_cast<int64_t>(pos) * d.rot_dim + 8 * g;
    load8f(cs, c);
    load8f(cs + (d.rot_dim >> 1), s);
  }
  const uint16_t* q = static_cast<const uint16_t*>(d.q) + t * d.q_token_ld;
  uint16_t* o = static_cast<uint16_t*>(d.q_out) + t * d.qo_token_ld;
  // four heads' loads before the first store: q_out may be q, so the compiler keeps
  // loads and stores in order (each thread rewrites only what it has read)
  constexpr int kAtOnce = 4;
  for (int h = h0; h < h1; h += kAtOnce) {
    uint4 u[kAtOnce], v[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (h + k < h1) {
        u[k] = *reinterpret_cast<const uint4*>(q + (h + k) * d.q_head_ld + ra);
        v[k] = *reinterpret_cast<const uint4*>(q + (h + k) * d.q_head_ld + rb);
      }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (h + k < h1) {
        if (turned) {
          float x[8], y[8];
          unpack8<F16>(u[k], x);
          unpack8<F16>(v[k], y);
          turn(x, y, c, s, inter);
          u[k] = pack8<F16>(x);
          v[k] = pack8<F16>(y);
        }
        *reinterpret_cast<uint4*>(o + (h + k) * d.qo_head_ld + ra) = u[k];
        *reinterpret_cast<uint4*>(o + (h + k) * d.qo_head_ld + rb) = v[k];
      }
  }
}

// What a unit's CTA has to do: the page's new slots and where their rows are.
struct PageWork {
  int b, pi, page, s0, s1;   // sequence, its page number, page, slots [s0, s1) of the new tokens
  int64_t row0;              // token row of slot 0
};

// Units are numbered so that sequence b's start at cu[b] / P + 2b: as many as it
// can need wherever its first token falls in a page, with no prefix sum.  False if
// the unit has nothing to do (faults are told).
__device__ __forceinline__ bool page_work(const moe_kv_append_desc& d, int unit, PageWork& w) {
  const moe_kv_cache& kc = d.cache;
  const int P = kc.page_size;
  w.b = warp_find(kc.batch, unit, [&](int i) { return __ldg(kc.cu_new + i) / P + 2 * i; });
  const int c0 = __ldg(kc.cu_new + w.b), c1 = __ldg(kc.cu_new + w.b + 1), len = __ldg(kc.kv_len + w.b);
  const int n = c1 - c0;
  if (n == 0) return false;
  if (const int32_t fault = sequence_fault(d, c0, c1, len)) {
    if (threadIdx.x == 0) set_err(d.err, fault);
    return false;
  }
  const int pos0 = len - n;                                  // position of the sequence's first new token
  const int nth = unit - (c0 / P + 2 * w.b);                 // of the pages the new tokens fall on
  w.pi = pos0 / P + nth;
  if (nth < 0 || w.pi > (len - 1) / P) return false;
  w.page = __ldg(kc.page_table + w.b * kc.table_ld + w.pi);
  w.s0 = max(pos0 - w.pi * P, 0);
  w.s1 = min(len - w.pi * P, P);
  w.row0 = c0 + (w.pi * P - pos0);
  if (w.page < 0 || w.page >= kc.pages || (d.rot_dim && w.pi * P + w.s1 > d.max_pos)) {
    if (threadIdx.x == 0) set_err(d.err, MOE_DEV_BAD_INDEX);
    return false;
  }
  return true;
}

// 16 codes of a slot that was there before, under the page's new scale.
__device__ __forceinline__ void rescale16(uint4* o, float before, float s, bool pow2) {
  const uint4 u = *o;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint2 q[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p = e4m3x2_to_f16x2(static_cast<uint16_t>(w[2 * half + (i >> 1)] >> (16 * (i & 1))));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p));
      f[2 * i] = v.x * before;
      f[2 * i + 1] = v.y * before;
    }
    q[half] = codes8(f, s, pow2);
  }
  *o = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
}

// A row's 16 values of group g, rotated.
template <bool F16>
__device__ __forceinline__ void rotated16(const uint4& u, const uint4& v, const float* cos_sin, int pos, int g, int rot, bool inter,
                                          float (&x)[8], float (&y)[8]) {
  unpack8<F16>(u, x);
  unpack8<F16>(v, y);
  if (g < (rot >> 4)) {
    float c[8], s[8];
    const float* cs = cos_sin + static_cast<int64_t>(pos) * rot + 8 * g;
    load8f(cs, c);
    load8f(cs + (rot >> 1), s);
    turn(x, y, c, s, inter);
  }
}

// A page's scale from the maximum of its new tokens; whether old codes have to follow.
__device__ __forceinline__ float page_scale(float amax, bool joins, float before, bool& grown, bool& pow2) {
  uint8_t byte;
  float s = block_scale_ue8m0(amax, &byte);
  grown = joins && s > before;
  if (joins && !grown) s = before;
  pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
  return s;
}

template <bool F16, int D>
__global__ void __launch_bounds__(128) kv_append_tokens_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int TT = 128, kGroups = D / 16;
  const moe_kv_append_desc& d = a.d;
  const moe_kv_cache& kc = d.cache;
  grid_dependency_wait();
  grid_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= a.kv_ctas) {
    const int cta = blockIdx.x - a.kv_ctas;
    if (cta < a.q_ctas) rotate_queries<F16, D, TT>(a, cta); else check_offsets<TT>(d, cta - a.q_ctas);
    return;
  }
  PageWork w;
  if (!page_work(d, blockIdx.x, w)) return;
  const bool inter = (d.flags & MOE_KV_INTERLEAVED) != 0;
  const int P = kc.page_size, g = threadIdx.x % kGroups;
  // rows of (K or V, head), kGroups lanes to each; whole groups of lanes take part or not
  for (int row = threadIdx.x / kGroups; row < 2 * kc.kv_heads; row += TT / kGroups) {
    const bool is_v = row >= kc.kv_heads;
    const int h = is_v ? row - kc.kv_heads : row, rot = is_v ? 0 : d.rot_dim;
    const int64_t tld = is_v ? d.v_token_ld : d.k_token_ld, sld = is_v ? kc.v_slot_ld : kc.k_slot_ld;
    int ra, rb;
    group_runs(g, rot, inter, ra, rb);
    const uint16_t* src = static_cast<const uint16_t*>(is_v ? d.v : d.k) + w.row0 * tld + h * (is_v ? d.v_head_ld : d.k_head_ld);
    uint8_t* out = is_v ? kc.v + w.page * kc.v_page_ld + h * kc.v_head_ld : kc.k + w.page * kc.k_page_ld + h * kc.k_head_ld;
    float* scale = (is_v ? kc.v_scale : kc.k_scale) + static_cast<int64_t>(w.page) * kc.kv_heads + h;
    const float before = w.s0 > 0 ? *scale : 0.0f;
    float x[8], y[8], amax = 0.0f;
    // four slots' loads at once: a sequence of the batch may have many new tokens after all
    constexpr int kAtOnce = 4;
    uint4 u[kAtOnce], v[kAtOnce];
    const auto load = [&](int slot) {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (slot + k < w.s1) {
          const uint16_t* p = src + (slot + k) * tld;
          u[k] = __ldg(reinterpret_cast<const uint4*>(p + ra));
          v[k] = __ldg(reinterpret_cast<const uint4*>(p + rb));
        }
    };
    const uint32_t lanes = kGroups == 8 ? 0xFFu << (threadIdx.x & 24) : 0xFu << (threadIdx.x & 28);
    for (int finite = 0; finite < 2; ++finite) {
      amax = 0.0f;
      for (int slot = w.s0; slot < w.s1; slot += kAtOnce) {
        load(slot);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (slot + k < w.s1) {
            rotated16<F16>(u[k], v[k], d.cos_sin, w.pi * P + slot + k, g, rot, inter, x, y);
            amax = finite ? finite_max(x, y, amax) : abs_max(x, y, amax);
          }
      }
#pragma unroll
      for (int o = 1; o < kGroups; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
      if (amax <= FLT_MAX) break;          // nearly always
    }
    bool grown, pow2;
    const float s = page_scale(amax, w.s0 > 0, before, grown, pow2);
    for (int slot = w.s0; slot < w.s1; slot += kAtOnce) {
      if (w.s1 - w.s0 > kAtOnce) load(slot);             // else they are still in registers
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (slot + k < w.s1) {
          rotated16<F16>(u[k], v[k], d.cos_sin, w.pi * P + slot + k, g, rot, inter, x, y);
          uint8_t* o = out + (slot + k) * sld;
          *reinterpret_cast<uint2*>(o + ra) = codes8(x, s, pow2);
          *reinterpret_cast<uint2*>(o + rb) = codes8(y, s, pow2);
        }
    }
    if (grown)
      for (int slot = 0; slot < w.s0; ++slot) rescale16(reinterpret_cast<uint4*>(out + slot * sld + 16 * g), before, s, pow2);
    if (g == 0) *scale = s;
  }
}

// CTAs of the pages kernel that share an SM (its registers are limited to that).
template <int TT, int R>
constexpr int kPagesPerSm = R == 1 ? 1024 / TT : 1;

template <bool F16, int D, int TT, int R>
__global__ void __launch_bounds__(TT, kPagesPerSm<TT, R>) kv_append_pages_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ uint32_t red[3][TT / 32];
  const moe_kv_append_desc& d = a.d;
  const moe_kv_cache& kc = d.cache;
  grid_dependency_wait();
  grid_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= a.kv_ctas) {
    check_offsets<TT>(d, blockIdx.x - a.kv_ctas);
    return;
  }
  constexpr int kGroups = D / 16;
  const int P = kc.page_size;
  const int hg = blockIdx.x % a.head_groups;
  const bool is_v = (blockIdx.x / a.head_groups) & 1;
  PageWork w;
  if (!page_work(d, blockIdx.x / (2 * a.head_groups), w)) return;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? d.v : d.k);
  const int64_t src_tld = is_v ? d.v_token_ld : d.k_token_ld, src_hld = is_v ? d.v_head_ld : d.k_head_ld;
  uint8_t* dst = (is_v ? kc.v + w.page * kc.v_page_ld : kc.k + w.page * kc.k_page_ld);
  const int64_t dst_hld = is_v ? kc.v_head_ld : kc.k_head_ld, dst_sld = is_v ? kc.v_slot_ld : kc.k_slot_ld;
  float* scale = (is_v ? kc.v_scale : kc.k_scale) + static_cast<int64_t>(w.page) * kc.kv_heads;
  const int rot = is_v ? 0 : d.rot_dim;
  const bool inter = (d.flags & MOE_KV_INTERLEAVED) != 0;
  const int h0 = hg * a.heads_per, h1 = min(h0 + a.heads_per, kc.kv_heads);

  uint4 u[R], v[R];
  const auto load = [&](int h) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int item = threadIdx.x + r * TT;
      const int slot = item / kGroups, g = item % kGroups;
      int ra, rb;
      group_runs(g, rot, inter, ra, rb);
      if (slot >= w.s0 && slot < w.s1) {
        const uint16_t* p = src + (w.row0 + slot) * src_tld + h * src_hld;
        u[r] = __ldg(reinterpret_cast<const uint4*>(p + ra));
        v[r] = __ldg(reinterpret_cast<const uint4*>(p + rb));
      } else {
        u[r] = v[r] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  load(h0);
  for (int h = h0; h < h1; ++h) {
    float x[R][8], y[R][8];
    float amax = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int item = threadIdx.x + r * TT;
      const int slot = item / kGroups, g = item % kGroups;
      const bool in = slot >= w.s0 && slot < w.s1;
      rotated16<F16>(u[r], v[r], d.cos_sin, w.pi * P + (in ? slot : w.s0), g, rot, inter, x[r], y[r]);
      amax = abs_max(x[r], y[r], amax);                // rows that are none are zeros
    }
    const float before = scale[h];
    if (h + 1 < h1) load(h + 1);
    // over the CTA: floats that are not negative order as their bit patterns do
    const auto all_max = [&](float m, uint32_t* slots) {
      const uint32_t wmax = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
      if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = wmax;
      __syncthreads();
      uint32_t all = 0;
#pragma unroll
      for (int k = 0; k < TT / 32; ++k) all = max(all, slots[k]);
      return __uint_as_float(all);
    };
    amax = all_max(amax, red[h & 1]);
    if (amax > FLT_MAX) {                  // an infinity among them
      amax = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r) amax = finite_max(x[r], y[r], amax);
      amax = all_max(amax, red[2]);
      __syncthreads();                     // red[2] may be used again
    }
    bool grown, pow2;
    const float s = page_scale(amax, w.s0 > 0, before, grown, pow2);
    uint8_t* out = dst + h * dst_hld;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int item = threadIdx.x + r * TT;
      const int slot = item / kGroups, g = item % kGroups;
      if (slot < w.s0 || slot >= w.s1) continue;
      int ra, rb;
      group_runs(g, rot, inter, ra, rb);
      uint8_t* o = out + slot * dst_sld;
      *reinterpret_cast<uint2*>(o + ra) = codes8(x[r], s, pow2);
      *reinterpret_cast<uint2*>(o + rb) = codes8(y[r], s, pow2);
    }
    if (grown)
      for (int item = threadIdx.x; item < w.s0 * kGroups; item += TT)
        rescale16(reinterpret_cast<uint4*>(out + item / kGroups * dst_sld + 16 * (item % kGroups)), before, s, pow2);
    // every thread read the old scale before the barrier above
    if (threadIdx.x == 0) scale[h] = s;
  }
}

template <bool F16, int D>
__global__ void __launch_bounds__(256, 3) kv_rotate_queries_kernel(const __grid_constant__ AppendArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  rotate_queries<F16, D, 256>(a, blockIdx.x);
}

// How many CTAs the queries take, TT threads each.
template <int D, int TT>
int64_t query_ctas(AppendArgs& a) {
  constexpr int kRows = TT / (D / 16);
  a.q_groups = (a.d.q_heads + kQHeadsPerCta - 1) / kQHeadsPerCta;
  return a.d.q ? (a.d.T + kRows - 1) / kRows * a.q_groups : 0;
}

template <bool F16, int D, int TT, int R>
int launch_pages(AppendArgs& a, cudaStream_t st) {
  // several heads a CTA, so that a page's chain of loads is paid once for them, as long
  // as there is a CTA for every place on the GPU (32768 prompt
  // tokens' keys and values: 56 us)
  const int64_t heads = a.d.cache.kv_heads, per = 2 * a.units * heads / (kPagesPerSm<TT, R> * num_sms());
  a.head_groups = static_cast<int32_t>(per <= 1 ? heads : (heads + per - 1) / per);
  a.heads_per = static_cast<int32_t>((heads + a.head_groups - 1) / a.head_groups);
  const int64_t kv = 2ll * a.units * a.head_groups, qc = query_ctas<D, 256>(a), all = kv + check_ctas<TT>(a);
  if (all > INT32_MAX || qc > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  a.kv_ctas = static_cast<int32_t>(kv);
  if (int rc = launch_pdl(kv_append_pages_kernel<F16, D, TT, R>, dim3(static_cast<unsigned>(all)), dim3(TT), 0, st, a)) return rc;
  if (qc == 0) return MOE_OK;
  return launch_pdl(kv_rotate_queries_kernel<F16, D>, dim3(static_cast<unsigned>(qc)), dim3(256), 0, st, a);
}

template <bool F16, int D>
int launch_tokens(AppendArgs& a, cudaStream_t st) {
  const int64_t qc = query_ctas<D, 128>(a), all = a.units + qc + check_ctas<128>(a);
  if (all > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  a.kv_ctas = a.units;
  a.q_ctas = static_cast<int32_t>(qc);
  return launch_pdl(kv_append_tokens_kernel<F16, D>, dim3(static_cast<unsigned>(all)), dim3(128), 0, st, a);
}

// One thread holds 16 values of a row, so a page takes page_size * dim / 16
// threads, or half as many with two rows each above 512.
template <bool F16>
int pick_append(AppendArgs& a, cudaStream_t st) {
  const int P = a.d.cache.page_size;
  a.units = static_cast<int32_t>(a.d.T / P) + 2 * a.d.cache.batch;
  // few new tokens a sequence: all heads of a page in one CTA (see the kernels)
  if (a.d.T <= kFewTokens * a.d.cache.batch) return a.d.cache.dim == 64 ? launch_tokens<F16, 64>(a, st) : launch_tokens<F16, 128>(a, st);
  if (a.d.cache.dim == 64) {
    if (P == 16) return launch_pages<F16, 64, 64, 1>(a, st);
    if (P == 32) return launch_pages<F16, 64, 128, 1>(a, st);
    if (P == 64) return launch_pages<F16, 64, 256, 1>(a, st);
    return launch_pages<F16, 64, 512, 1>(a, st);
  }
  if (P == 16) return launch_pages<F16, 128, 128, 1>(a, st);
  if (P == 32) return launch_pages<F16, 128, 256, 1>(a, st);
  if (P == 64) return launch_pages<F16, 128, 512, 1>(a, st);
  return launch_pages<F16, 128, 512, 2>(a, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_kv_append(const moe_kv_append_desc* d, void* stream) {
  MOE_CHECK_ARG(d != nullptr);
  if (int rc = check_kv_cache(d->cache, d->T)) return rc;
  MOE_CHECK_ARG((d->flags & ~MOE_KV_INTERLEAVED) == 0);
  MOE_CHECK_ARG(d->rot_dim >= 0 && d->rot_dim <= d->cache.dim && d->rot_dim % 16 == 0 && d->max_pos >= 0);
  MOE_CHECK_ARG(kv_strides_ok(d->k_token_ld, d->k_head_ld, d->v_token_ld, 8) &&
                kv_strides_ok(d->v_head_ld, d->q_token_ld, d->q_head_ld, 8) &&
                kv_strides_ok(d->qo_token_ld, d->qo_head_ld, 0, 8));
  if (d->T == 0 || d->cache.batch == 0) return MOE_OK;
  MOE_CHECK_ARG(d->k && d->v && aligned16(d->k) && aligned16(d->v));
  MOE_CHECK_ARG(d->rot_dim == 0 || (d->cos_sin && aligned16(d->cos_sin)));
  if (d->q != nullptr) {
    MOE_CHECK_ARG(d->q_out && aligned16(d->q) && aligned16(d->q_out));
    MOE_CHECK_ARG(d->q_heads >= 1);
    if (d->q_heads > 65536) return MOE_ERR_UNSUPPORTED;
  } else {
    MOE_CHECK_ARG(d->q_heads == 0 && d->q_out == nullptr);
  }
  if (int rc = check_device()) return rc;
  AppendArgs a{};
  a.d = *d;
  return d->cache.dtype == MOE_DTYPE_F16 ? pick_append<true>(a, as_stream(stream))
                                         : pick_append<false>(a, as_stream(stream));
}
