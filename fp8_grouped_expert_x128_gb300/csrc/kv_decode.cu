// Attention over the paged 8-bit cache for few rows per kv head (decode steps
// and draft tokens): memory bound, 2 * dim bytes for each key token and kv head.
//
// The keys of every (sequence, kv head) are cut into 64-token tiles; the tiles of
// all of them, in order, are split evenly over the CTAs of one resident wave, so
// lengths that differ and few sequences both keep all SMs loading.  A (sequence,
// kv head) that several CTAs share is joined by the last of them to finish, from
// the running maximum, sum and unnormalised output that each has left in the
// workspace; parts are added in the order of their keys, so results repeat bit
// for bit whichever CTA comes last.  More than 32 parts are joined in two levels.
//
// A warp takes 16 keys of a tile through a cp.async ring of its own (no barrier
// inside a CTA's loop).  Both products run transposed on mma.m16n8k16 f16, S^T =
// K Q^T and O^T = V^T P^T, with the rows as the n side: 8 rows cost no padding to
// 16, and K fragments are read straight from shared memory, the head's dimensions
// taken in the order in which a lane's bytes lie (Q is put in the same order).
// E4M3 widens exactly to f16 in one instruction per pair.  The V scale rides in
// the weight: w = exp2(s + log2 s_V - m), the sum takes w / s_V; m follows the largest
// score, and the size of s_V both ways.
//
// A step is some 420 instructions (560 with two groups of rows) with little parallelism
// inside a warp, so three or four CTAs share an SM (two: 253 us where three took 191).
// Measured by graph replay: 64 sequences of 2000 to 16400 tokens, 8 kv heads, 4 rows
// each, 193 us, 6.2 TB/s (92% of a copy's); four of 131072 tokens, 166 us (96%); one of
// 1010 tokens, 11 us: four dependent loads, the join's release and acquire, and its
// loads, about a microsecond each.
#include "kv_attention.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;                 // keys a warp takes at a time
constexpr int kTile = kStep * kWarps;
constexpr int kGroup = 32;                // parts joined at a time, one lane each
constexpr int kMaxParts = 1024;           // CTAs of a launch at most
static_assert(kMaxParts <= kGroup * kGroup, "two levels");
static_assert(3 * kMaxParts == kDecodeCounters, "counters of the three levels");

template <int D, int NT>
struct Cfg {
  // CTAs that share an SM (registers and shared memory are sized for them) and the
  // stages of each warp's ring: some 150 KB under way on an SM either way
  static constexpr int kCtasPerSm = D == 128 ? 3 : 4;
  static constexpr int kStages = D == 128 ? 4 : 6;
  static constexpr int kStageBytes = 2 * kStep * D;       // K, then V
  static constexpr int kRows = 8 * NT;
  static constexpr int kLd = D + 4;                       // merge buffer row, padded against bank conflicts
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kScales = kRing;                   // [warp][stage][2] floats
  static constexpr int kBuf = kScales + kWarps * kStages * 8;
  static constexpr bool kSharedQ = NT > 1;                // Q's fragments: in registers for 8 rows, else shared
  static constexpr int kQ = kBuf;                         // [row / 8][16-deep step][lane] uint2, done with before buf is used
  static_assert(NT * (D / 16) * 256 <= kRows * kLd * 4, "Q fits where the merge buffer is");
  static constexpr int kSmem = kBuf + kRows * kLd * 4;
};
constexpr int kPartRows = 16;                             // of a CTA, at most
constexpr int kPartFloats = kPartRows * (128 + 2);        // one part: m[16], l[16], O[16][dim]

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk ch of key row r in a stage: chunks are swapped
// around within 128 bytes so that both the fragment loads of K (a lane's own
// bytes of 8 rows) and the transposing loads of V (one chunk of 8 rows) touch
// every bank once.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
  if constexpr (D == 128) {
    return static_cast<uint32_t>(r * 128 + ((ch ^ (r & 7)) << 4));
  } else {
    return static_cast<uint32_t>((r >> 1) * 128 + (((((r & 1) << 2) | ch) ^ ((r >> 1) & 7)) << 4));
  }
}

// Tiles of a sequence's keys, from the one with the first key its first row sees, and
// the groups of rows that walk over them: a kv head with more rows than a CTA holds
// is read again for the others (from L2, as a rule: their CTAs run side by side).
struct Tiles {
  int first, count, groups;
};
__device__ __forceinline__ Tiles tiles_of(const AttnArgs& a, const Seq& s, int group_rows) {
  Tiles t{0, 0, 0};
  if (s.n == 0 || s.n * a.G > kDecodeRows) return t;
  t.first = first_key(a.d, s, 0) / kTile;
  t.count = (s.len + kTile - 1) / kTile - t.first;
  // the 8-row kernel is launched where no sequence has more
  t.groups = group_rows == 8 ? 1 : (s.n * a.G + group_rows - 1) / group_rows;
  return t;
}

// a / b for a >= 0, b > 0: in 32 bits where they fit, as they nearly always do.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// First unit of CTA c when W units are split over C CTAs.
__device__ __forceinline__ int64_t range_start(int64_t W, int c, int C) { return quotient(W * c, C); }
// The CTA that owns unit u: the largest c with range_start(c) <= u.
__device__ __forceinline__ int owner(int64_t u, int64_t W, int C) {
  return static_cast<int>(quotient((u + 1) * C + W - 1, W)) - 1;
}

template <bool F16, int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtasPerSm) kv_decode_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<D, NT>;
  constexpr int KS = D / 16;              // 16-deep steps of S, and 16-dimension blocks of O
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[kWarps];
  __shared__ int64_t s_u;                 // units before the sequence that holds this CTA's first one
  __shared__ int s_b, s_last;
  __shared__ __align__(8) float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows], s_inv[C::kRows], s_qs[C::kRows];
  __shared__ __align__(8) int s_lo[C::kRows], s_hi[C::kRows];          // keys that a row sees

  const moe_kv_attention_desc& d = a.d;
  const moe_kv_cache& kc = d.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int H = kc.kv_heads, P = kc.page_size;
  const int page_shift = 31 - __clz(P);
  int ctas = gridDim.x;
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- this CTA's range of units, and the sequence it begins in: a scan over the sequences
  int64_t total, u0, u1, first_u;          // first_u: units before that sequence
  int first_b;
  int32_t bad = 0;
  const auto units_of = [&](int b) {
    const Tiles x = tiles_of(a, load_seq(d, b, &bad), C::kRows);
    return static_cast<int64_t>(x.count) * H * x.groups;
  };
  const auto inclusive = [&](int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    return v;
  };
  const auto my_range = [&] {
    // at least one unit each: the CTAs that share a row are then a run without gaps
    ctas = static_cast<int>(min(static_cast<int64_t>(ctas), total));
    u0 = u1 = 0;
    if (static_cast<int>(blockIdx.x) >= ctas) return;
    u0 = range_start(total, blockIdx.x, ctas);
    u1 = range_start(total, blockIdx.x + 1, ctas);
  };
  if (kc.batch <= 32) {
    // a lane for each, every warp for itself: no barrier (one sequence of 1010 tokens
    // 12.3 -> 11.5 us)
    const int64_t own = lane < kc.batch ? units_of(lane) : 0, incl = inclusive(own);
    total = __shfl_sync(0xffffffffu, incl, 31);
    my_range();
    first_b = __ffs(__ballot_sync(0xffffffffu, u0 < incl)) - 1;
    first_u = __shfl_sync(0xffffffffu, incl - own, max(first_b, 0));
  } else {                                 // a run of them for each thread
    const int per = (kc.batch + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, kc.batch), b1 = min(b0 + per, kc.batch);
    int64_t own = 0;
    for (int b = b0; b < b1; ++b) own += units_of(b);
    int64_t incl = inclusive(own);
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += scan[w];
      total += scan[w];
    }
    my_range();
    if (u0 >= incl - own && u0 < incl) {
      int64_t u = incl - own;
      for (int b = b0; b < b1; ++b) {
        const int64_t t = units_of(b);
        if (u0 < u + t) {
          s_b = b;
          s_u = u;
          break;
        }
        u += t;
      }
    }
    __syncthreads();
    first_b = s_b;
    first_u = s_u;
  }
  if (bad && blockIdx.x == 0) set_err(d.err, bad);
  if (u0 == u1) return;

  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
  float* ring_scales = reinterpret_cast<float*>(smem + C::kScales) + warp * C::kStages * 2;
  float* buf = reinterpret_cast<float*>(smem + C::kBuf);

  // ---- the first (sequence, kv head), and its queries on their way
  int32_t ignored = 0;                     // the scan has told
  int b = first_b;
  Seq s = load_seq(d, b, &ignored);
  Tiles t = tiles_of(a, s, C::kRows);
  int hg = static_cast<int>(quotient(u0 - first_u, t.count));          // kv head x group of rows
  int tile = t.first + static_cast<int>(u0 - first_u - static_cast<int64_t>(hg) * t.count);
  uint4 qw[D / 32];                        // lane (g, c): a quarter of row g (of 8 rows a warp where they are shared)
  const auto load_q = [&] {
    const int h = hg / t.groups, r = hg % t.groups * C::kRows + (C::kSharedQ ? warp * 8 : 0) + g;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) qw[k] = make_uint4(0, 0, 0, 0);
    if (r < s.n * a.G) {
      const int i = r / a.G;
      const uint16_t* qp = static_cast<const uint16_t*>(d.q) + (s.c0 + i) * d.q_token_ld + (h * a.G + r - i * a.G) * d.q_head_ld +
                           c * (D / 4);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) qw[k] = __ldg(reinterpret_cast<const uint4*>(qp) + k);
    }
  };
  load_q();

  // ---- producer: walks the CTA's units, kStages - 1 ahead of the consumer
  int64_t p_left = u1 - u0;
  int p_b = first_b, p_h, p_hg, p_tile, p_end, p_base, p_stage = 0, p_pid = 0;
  Seq p_s = s;
  Tiles p_t = t;
  // this lane's share of a step's copy: chunk ch of rows r, r + kRowsPer, ...
  constexpr int kChunks = D / 16, kRowsPer = 32 / kChunks;
  const int ld_r = lane / kChunks, ld_ch = lane % kChunks;
  const int64_t k_lane = ld_r * kc.k_slot_ld + ld_ch * 16, v_lane = ld_r * kc.v_slot_ld + ld_ch * 16;
  const auto p_pages = [&] {               // the page of this warp's keys in 32 tiles from p_tile, one per lane
    p_base = p_tile;
    const int key = (p_tile + lane) * kTile + warp * kStep;
    p_pid = key < p_s.len ? __ldg(kc.page_table + p_b * kc.table_ld + (key >> page_shift)) : 0;
  };
  p_hg = hg;
  p_h = hg / t.groups;
  p_tile = tile;
  p_end = t.first + t.count;
  p_pages();
  const auto issue = [&] {
    if (p_left > 0) {
      if (p_tile == p_end) {
        if (++p_hg == H * p_t.groups) {
          p_hg = 0;
          do {
            p_s = load_seq(d, ++p_b, &ignored);
            p_t = tiles_of(a, p_s, C::kRows);
          } while (p_t.count == 0 && p_b + 1 < kc.batch);
        }
        p_h = p_hg / p_t.groups;
        p_tile = p_t.first;
        p_end = p_t.first + p_t.count;
        p_pages();
      } else if (p_tile - p_base == 32) {
        p_pages();
      }
      const int key0 = p_tile * kTile + warp * kStep;
      int page = __shfl_sync(0xffffffffu, p_pid, p_tile - p_base);
      bool on = key0 < p_s.len;
      if (on && (page < 0 || page >= kc.pages)) {
        if (lane == 0) set_err(d.err, MOE_DEV_BAD_INDEX);
        on = false;
      }
      if (!on) page = 0;
      const int slot0 = key0 & (P - 1);
      const uint8_t* kp = kc.k + page * kc.k_page_ld + p_h * kc.k_head_ld + slot0 * kc.k_slot_ld + k_lane;
      const uint8_t* vp = kc.v + page * kc.v_page_ld + p_h * kc.v_head_ld + slot0 * kc.v_slot_ld + v_lane;
      const uint32_t st = ring + p_stage * C::kStageBytes;
      if (on && key0 + kStep <= p_s.len) {
#pragma unroll
        for (int i = 0; i < kStep / kRowsPer; ++i) {
          const uint32_t at = st + chunk_at<D>(ld_r + i * kRowsPer, ld_ch);
          cp16(at, kp, true);
          cp16(at + kStep * D, vp, true);
          kp += kRowsPer * kc.k_slot_ld;
          vp += kRowsPer * kc.v_slot_ld;
        }
      } else {                             // past the end: zeros, nothing is read
#pragma unroll
        for (int i = 0; i < kStep / kRowsPer; ++i) {
          const uint32_t at = st + chunk_at<D>(ld_r + i * kRowsPer, ld_ch);
          const bool in = on && key0 + ld_r + i * kRowsPer < p_s.len;
          cp16(at, in ? kp : kc.k, in);
          cp16(at + kStep * D, in ? vp : kc.v, in);
          kp += kRowsPer * kc.k_slot_ld;
          vp += kRowsPer * kc.v_slot_ld;
        }
      }
      if (lane < 2) {
        const float* sp = (lane ? kc.v_scale : kc.k_scale) + static_cast<int64_t>(page) * H + p_h;
        cp_async_4(smem_u32(ring_scales + p_stage * 2 + lane), sp, on ? 4 : 0);
      }
      ++p_tile;
      --p_left;
      if (++p_stage == C::kStages) p_stage = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages - 1; ++i) issue();

  // ---- consumer: one (sequence, kv head) after the other
  int stage = 0;
  int64_t u = u0;
  while (true) {
    const int h = hg / t.groups, row0 = hg % t.groups * C::kRows;
    const int rows = min(C::kRows, s.n * a.G - row0);        // of this group, from row0 on
    const int tile_begin = tile;
    const int tile_stop = static_cast<int>(min(static_cast<int64_t>(t.first + t.count), tile + (u1 - u)));
    const int lo_first = first_key(d, s, row0 / a.G), lo_last = first_key(d, s, (row0 + rows - 1) / a.G);
    const int hi_first = end_key(d, s, row0 / a.G), hi_last = end_key(d, s, (row0 + rows - 1) / a.G);

    // Q as the second operand: lane (g, c) holds row g's dimensions c * D/4 ..., scaled into f16
    uint32_t q[C::kSharedQ ? 1 : KS][2];
    float qs[C::kSharedQ ? 1 : 2], m[NT][2], l[NT][2], o[NT][KS][4];
    uint2* s_q = reinterpret_cast<uint2*>(smem + C::kQ);
    if (tid < C::kRows) {
      const int i = min((row0 + tid) / a.G, s.n - 1);
      s_lo[tid] = first_key(d, s, i);
      s_hi[tid] = end_key(d, s, i);
    }
    if (!C::kSharedQ || warp < NT) {
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        float f[8];
        unpack8<F16>(qw[k], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = f[e] != f[e] ? INFINITY : fmaxf(amax, fabsf(f[e]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float mul, inv;
      row_scale(amax, mul, inv);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        float f[8];
        unpack8<F16>(qw[k], f);
        const uint2 x = make_uint2(f16x2(f[0] * mul, f[1] * mul), f16x2(f[2] * mul, f[3] * mul));
        const uint2 y = make_uint2(f16x2(f[4] * mul, f[5] * mul), f16x2(f[6] * mul, f[7] * mul));
        if constexpr (C::kSharedQ) {
          s_q[(warp * KS + 2 * k) * 32 + lane] = x;
          s_q[(warp * KS + 2 * k + 1) * 32 + lane] = y;
        } else {
          q[2 * k][0] = x.x; q[2 * k][1] = x.y;
          q[2 * k + 1][0] = y.x; q[2 * k + 1][1] = y.y;
        }
      }
      inv *= d.softcap > 0.0f ? d.sm_scale / d.softcap : d.sm_scale * kLog2e;
      if constexpr (C::kSharedQ) {
        if (c == 0) s_qs[warp * 8 + g] = inv;
      } else {
        qs[0] = __shfl_sync(0xffffffffu, inv, 8 * c);     // of the columns of S^T that this lane holds
        qs[1] = __shfl_sync(0xffffffffu, inv, 8 * c + 4);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][k][e] = 0.0f;
    }
    __syncthreads();

    uint32_t nan_seen = 0;
    float size = -INFINITY, largest = -INFINITY;   // logarithm of the V scales that m goes with; of the largest
#pragma unroll 1
    for (; tile < tile_stop; ++tile) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
      __syncwarp();
      const int key0 = tile * kTile + warp * kStep;
      if (key0 < hi_last && key0 + kStep > lo_first) {
        const uint32_t ks = ring + stage * C::kStageBytes, vs = ks + kStep * D;
        const float k_scale = ring_scales[stage * 2], v_scale = fmaxf(ring_scales[stage * 2 + 1], kMinScale);
        const float v_log = __log2f(v_scale), v_inv = __fdividef(1.0f, v_scale);
        const bool edge = key0 < lo_last || key0 + kStep > hi_first;
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = 0.0f;
#pragma unroll
        for (int k4 = 0; k4 < KS / 4; ++k4) {
          const int ch = c * (D / 64) + k4;
          const uint4 x = lds16(ks + chunk_at<D>(g, ch)), y = lds16(ks + chunk_at<D>(g + 8, ch));
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t f[4] = {e4m3x2_to_f16x2(xw[k] & 0xFFFF), e4m3x2_to_f16x2(yw[k] & 0xFFFF),
                                   e4m3x2_to_f16x2(xw[k] >> 16), e4m3x2_to_f16x2(yw[k] >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (nt == 0 || nt * 8 < rows) {
                if constexpr (C::kSharedQ) {
                  const uint2 x = s_q[(nt * KS + k4 * 4 + k) * 32 + lane];
                  mma(sc[nt], f, x.x, x.y);
                } else {
                  mma(sc[nt], f, q[k4 * 4 + k][0], q[k4 * 4 + k][1]);
                }
              }
          }
        }
        // scores in powers of two, with the V scale's logarithm
        float f[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (C::kSharedQ) {
            const float2 x = *reinterpret_cast<const float2*>(s_qs + nt * 8 + 2 * c);
            f[nt][0] = x.x * k_scale;
            f[nt][1] = x.y * k_scale;
          } else {
            f[nt][0] = qs[0] * k_scale;
            f[nt][1] = qs[1] * k_scale;
          }
        }
        if (d.softcap > kCapDirect) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = sc[nt][e] * f[nt][e & 1];
              sc[nt][e] = fmaf(y * tanh_ratio(y), d.softcap * kLog2e, v_log);
            }
        } else if (d.softcap > 0.0f) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[nt][e] = capped_log2(sc[nt][e] * f[nt][e & 1], d.softcap * kLog2e) + v_log;
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][e] = fmaf(sc[nt][e], f[nt][e & 1], v_log);
        }
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int2 lo = *reinterpret_cast<const int2*>(s_lo + nt * 8 + 2 * c);
            const int2 hi = *reinterpret_cast<const int2*>(s_hi + nt * 8 + 2 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + g + (e >> 1) * 8;
              if (key < (e & 1 ? lo.y : lo.x) || key >= (e & 1 ? hi.y : hi.x)) sc[nt][e] = -INFINITY;
            }
          }
        }
        bool over = fabsf(v_log - size) > kNear;           // another size of V: the same for the warp
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          over |= fmaxf(sc[nt][0], sc[nt][2]) > m[nt][0] + kLazy || fmaxf(sc[nt][1], sc[nt][3]) > m[nt][1] + kLazy;
        if (__any_sync(0xffffffffu, over)) {
          // The reference goes with the size of the V scales, down as well as up, so that the
          // weights are as precise as before; fp32 holds what there is (but not below 2^-60 of
          // the largest, where it might not).  Then it goes with the maximum.
          float by = 0.0f;
          if (fabsf(v_log - size) > kNear) {
            largest = fmaxf(largest, v_log);
            const float to = fmaxf(v_log, largest - 60.0f);
            if (size > -INFINITY) by = to - size;
            size = to;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(sc[nt][e], sc[nt][e + 2]);
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              x = fmaxf(x - kHead, m[nt][e] + by);
              const float keep = x == -INFINITY ? 1.0f : ex2(m[nt][e] - x);
              m[nt][e] = x;
              l[nt][e] *= keep;
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                o[nt][k][e] *= keep;
                o[nt][k][e + 2] *= keep;
              }
            }
        }
        uint32_t p[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = ex2(sc[nt][e] - (m[nt][e & 1] == -INFINITY ? 0.0f : m[nt][e & 1]));
          l[nt][0] = fmaf(w[0] + w[2], v_inv, l[nt][0]);
          l[nt][1] = fmaf(w[1] + w[3], v_inv, l[nt][1]);
          p[nt][0] = transposed(f16x2(w[0], w[1]));
          p[nt][1] = transposed(f16x2(w[2], w[3]));
        }
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) {
          uint32_t v[4];
          ldsm4_t(vs + chunk_at<D>((lane & 7) + (lane & 8), 2 * k2 + (lane >> 4)), v);
          if (edge) {
            // a NaN that some row does not see must not meet its zero weight: it is
            // put back for the rows that do see it once the keys are done
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t bad = nan_codes(v[i]);
              nan_seen |= bad;
              v[i] &= ~((bad >> 7) * 0xFFu);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = __byte_perm(v[2 * i], 0, 0x3120), y = __byte_perm(v[2 * i + 1], 0, 0x3120);
            const uint32_t f[4] = {e4m3x2_to_f16x2(x & 0xFFFF), e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y & 0xFFFF),
                                   e4m3x2_to_f16x2(y >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (nt == 0 || nt * 8 < rows) mma(o[nt][2 * k2 + i], f, p[nt][0], p[nt][1]);
          }
        }
      }
      __syncwarp();                        // every lane has read the stage that is filled next
      issue();
      if (++stage == C::kStages) stage = 0;
    }

    // ---- the four warps' results together, in buf: m, l and the unnormalised output
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
        if (g == 0) {
          s_m[warp][nt * 8 + 2 * c + e] = m[nt][e];
          s_l[warp][nt * 8 + 2 * c + e] = l[nt][e];
        }
      }
    const bool fix_nan = __syncthreads_or(nan_seen != 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * c + e;
        float top = s_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
        // a warp without weights (m = -inf) may still hold a NaN
        const float keep = m[nt][e] == -INFINITY ? 1.0f : ex2(m[nt][e] - top);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          o[nt][k][e] *= keep;
          o[nt][k][e + 2] *= keep;
        }
      }
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (warp == w) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float2* at = reinterpret_cast<float2*>(buf + (nt * 8 + 2 * c + e) * C::kLd + 16 * k + 2 * g);
              float2 x = w ? *at : make_float2(0.0f, 0.0f);
              x.x += o[nt][k][e];
              x.y += o[nt][k][e + 2];
              *at = x;
            }
      }
      __syncthreads();
    }
    float top = -INFINITY, sum = 0.0f;     // of row tid
    if (tid < C::kRows) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        sum += s_l[w][tid] * (s_m[w][tid] == -INFINITY ? 1.0f : ex2(s_m[w][tid] - top));
    }
    if (fix_nan) {
      for (int x = tid; x < rows * D; x += kThreads) {
        const int r = x / D, dim = x % D, i = (row0 + r) / a.G;
        const int from = max(first_key(d, s, i), tile_begin * kTile), to = min(end_key(d, s, i), tile_stop * kTile);
        for (int j = from; j < to; ++j) {
          const int k0 = j & ~(kStep - 1);
          if (!(k0 < lo_last || k0 + kStep > hi_first)) {   // not a step whose NaNs were taken out
            j = max(j, (hi_first & ~(kStep - 1)) - 1);      // on to the next one
            continue;
          }
          const int page = __ldg(kc.page_table + b * kc.table_ld + (j >> page_shift));
          if (page < 0 || page >= kc.pages) continue;
          const uint8_t code = kc.v[page * kc.v_page_ld + h * kc.v_head_ld + (j & (P - 1)) * kc.v_slot_ld + dim];
          if ((code & 0x7F) == 0x7F) buf[r * C::kLd + dim] = __uint_as_float(0x7FC00000u);
        }
      }
      __syncthreads();
    }

    // ---- write the rows, or leave a part and let the last CTA join them
    const int64_t seg0 = u - (tile_begin - t.first), seg1 = seg0 + t.count;   // units of this (sequence, kv head)
    const bool whole = seg0 >= u0 && seg1 <= u1;
    const auto write_rows = [&] {
      if (tid < C::kRows) {
        s_inv[tid] = sum == 0.0f ? 0.0f : 1.0f / sum;       // NaN stays
        if (d.lse != nullptr && tid < rows) {
          const int i = (row0 + tid) / a.G;
          d.lse[static_cast<int64_t>(s.c0 + i) * d.q_heads + h * a.G + row0 + tid - i * a.G] =
              sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
        }
      }
      __syncthreads();
      for (int x = tid; x < rows * (D / 8); x += kThreads) {
        const int r = x / (D / 8), e = x % (D / 8) * 8, i = (row0 + r) / a.G;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = buf[r * C::kLd + e + k] * s_inv[r];
        uint16_t* op = static_cast<uint16_t*>(d.out) + (s.c0 + i) * d.o_token_ld + (h * a.G + row0 + r - i * a.G) * d.o_head_ld + e;
        *reinterpret_cast<uint4*>(op) = pack8<F16>(f);
      }
    };
    if (whole) {
      write_rows();
    } else {
      const int ca = owner(seg0, total, ctas), cz = owner(seg1 - 1, total, ctas);
      // a CTA leaves at most two parts: of a row that began before it, and of one that goes on after it
      const auto part_of = [&](int cta) { return a.parts + (2ll * cta + (cta == ca ? 1 : 0)) * kPartFloats; };
      const auto leave = [&](float* part) {
        if (tid < rows) {
          __stcg(part + tid, top);
          __stcg(part + kPartRows + tid, sum);
        }
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
          const int r = x / (D / 4), e = x % (D / 4) * 4;
          __stcg(reinterpret_cast<float4*>(part + 2 * kPartRows + r * D + e),
                 *reinterpret_cast<const float4*>(buf + r * C::kLd + e));
        }
      };
      // The barrier orders the CTA's stores before thread 0's release, and its acquire
      // before their loads.
      const auto arrive_last = [&](int32_t* counter, int count) {
        __syncthreads();
        if (tid == 0) {
          int before;
          asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
          s_last = before == count - 1;
          if (s_last) *counter = 0;                          // as the next call wants it
        }
        __syncthreads();
        return s_last != 0;
      };
      // parts of CTAs first, first + stride, ... into buf, top and sum
      const auto join = [&](int first, int stride, int count) {
        for (int r = warp; r < rows; r += kWarps) {
          const float* part = part_of(first + min(lane, count - 1) * stride);
          const float pm = lane < count ? __ldcg(part + r) : -INFINITY;
          float pl = lane < count ? __ldcg(part + kPartRows + r) : 0.0f, pt = pm;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) pt = fmaxf(pt, __shfl_xor_sync(0xffffffffu, pt, o));
          pl *= pm == -INFINITY ? 1.0f : ex2(pm - pt);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) pl += __shfl_xor_sync(0xffffffffu, pl, o);
          if (lane == 0) {
            s_m[0][r] = pt;
            s_l[0][r] = pl;
          }
        }
        __syncthreads();
        if (tid < rows) {
          top = s_m[0][tid];
          sum = s_l[0][tid];
        }
        // some 16 loads a thread under way; rows that are none load the last one's
        constexpr int kItems = C::kRows * (D / 4) / kThreads, kAtOnce = kItems >= 8 ? 2 : 16 / kItems;
        float4 acc[kItems];
#pragma unroll
        for (int y = 0; y < kItems; ++y) acc[y] = make_float4(0, 0, 0, 0);
#pragma unroll 1
        for (int k0 = 0; k0 < count; k0 += kAtOnce) {
          float pm[kAtOnce][kItems];
          float4 v[kAtOnce][kItems];
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            const float* part = part_of(first + min(k0 + k, count - 1) * stride);
#pragma unroll
            for (int y = 0; y < kItems; ++y) {
              const int r = min((tid + y * kThreads) / (D / 4), rows - 1), e = tid % (D / 4) * 4;
              pm[k][y] = __ldcg(part + r);
              v[k][y] = __ldcg(reinterpret_cast<const float4*>(part + 2 * kPartRows + r * D + e));
            }
          }
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
            for (int y = 0; y < kItems; ++y) {
              const int r = min((tid + y * kThreads) / (D / 4), rows - 1);
              float keep = pm[k][y] == -INFINITY ? 1.0f : ex2(pm[k][y] - s_m[0][r]);
              if (k0 + k < count) {
                acc[y].x = fmaf(v[k][y].x, keep, acc[y].x);
                acc[y].y = fmaf(v[k][y].y, keep, acc[y].y);
                acc[y].z = fmaf(v[k][y].z, keep, acc[y].z);
                acc[y].w = fmaf(v[k][y].w, keep, acc[y].w);
              }
            }
        }
#pragma unroll
        for (int y = 0; y < kItems; ++y) {
          const int r = (tid + y * kThreads) / (D / 4), e = tid % (D / 4) * 4;
          *reinterpret_cast<float4*>(buf + r * C::kLd + e) = acc[y];
        }
        __syncthreads();
      };
      // Counters: a CTA may be the first of the row it begins and of a later group
      // of the row it goes on with, so these count apart.
      const int parts = cz - ca + 1;
      leave(part_of(blockIdx.x));
      const int group = ca + (static_cast<int>(blockIdx.x) - ca) / kGroup * kGroup;
      const int in_group = min(kGroup, cz - group + 1);
      if (arrive_last(a.counters + (group == ca ? 0 : kMaxParts) + group, in_group)) {
        join(group, 1, in_group);
        if (parts <= kGroup) {
          write_rows();
        } else {
          // the group's first part takes the group's sum
          leave(part_of(group));
          const int groups = (parts + kGroup - 1) / kGroup;
          if (arrive_last(a.counters + 2 * kMaxParts + ca, groups)) {
            join(ca, kGroup, groups);
            write_rows();
          }
        }
      }
    }
    u += tile_stop - tile_begin;
    if (u >= u1) break;
    // the next (sequence, kv head)
    if (++hg == H * t.groups) {
      hg = 0;
      do {
        s = load_seq(d, ++b, &ignored);
        t = tiles_of(a, s, C::kRows);
      } while (t.count == 0 && b + 1 < kc.batch);
    }
    tile = t.first;
    load_q();
    __syncthreads();                       // buf and the statistics are free
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <bool F16, int D, int NT>
int launch(const AttnArgs& a, cudaStream_t st) {
  static int prepared[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  constexpr int smem = Cfg<D, NT>::kSmem;
  if (!__atomic_load_n(&prepared[dev], __ATOMIC_ACQUIRE)) {
    MOE_CUDA_TRY(cudaFuncSetAttribute(kv_decode_kernel<F16, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    __atomic_store_n(&prepared[dev], 1, __ATOMIC_RELEASE);
  }
  const int ctas = min(kMaxParts, num_sms() * Cfg<D, NT>::kCtasPerSm);
  return launch_pdl(kv_decode_kernel<F16, D, NT>, dim3(ctas), dim3(kThreads), smem, st, a);
}

template <bool F16, int D>
int pick_rows(const AttnArgs& a, int64_t rows, cudaStream_t st) {
  // 32 rows a CTA were measured too: their accumulators leave room for two CTAs an SM,
  // and 28 draft rows took 68 us against 65 with 16 rows a CTA and the keys read twice.
  return rows <= 8 ? launch<F16, D, 1>(a, st) : launch<F16, D, 2>(a, st);
}

}  // namespace

size_t kv_decode_workspace() {
  const size_t ctas = static_cast<size_t>(min(kMaxParts, num_sms() * 4));      // of the kernel with most
  return ctas * 2 * kPartFloats * sizeof(float);
}

int kv_decode_launch(const AttnArgs& a, int64_t max_rows, cudaStream_t st) {
  const bool f16 = a.d.cache.dtype == MOE_DTYPE_F16;
  if (a.d.cache.dim == 64) return f16 ? pick_rows<true, 64>(a, max_rows, st) : pick_rows<false, 64>(a, max_rows, st);
  return f16 ? pick_rows<true, 128>(a, max_rows, st) : pick_rows<false, 128>(a, max_rows, st);
}

}  // namespace moe
