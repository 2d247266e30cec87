// Attention over the paged 8-bit cache for many rows per kv head (prompts and
// chunks of prompts): bound by the tensor cores, 4 * dim operations for each row
// and visible key.
//
// A CTA takes 256 rows (new tokens x the query heads of one kv head, so that
// grouped heads fill tiles too) as two 128-row tiles, and walks over their keys, 64
// a step.  Per tile and step: S = Q K^T (tcgen05, f16, both operands in shared
// memory) into TMEM; a warpgroup, one row per thread, turns S into softmax weights
// and writes them back over S as f16; O += P V with P read from TMEM.  S has two
// buffers, so that a step's S is there when its softmax begins.  Two more
// warpgroups widen E4M3 K and V to f16 (exact), 128 keys at a time, on the way into
// shared memory, straight from global memory through registers, so pages and
// strides cost little; a warp for each tile issues its MMAs, and one more brings the page
// scales, which stay out of the operands: K's multiply the scores, V's ride in the weights
// as in the decode kernel.  Where there are fewer 256-row units than SMs, the keys are
// split as well, and kv_prefill_join_kernel adds the parts.
//
// Measured by graph replay: an 8192-token prompt with 64 / 8 heads of 128 in 0.965 ms,
// 1.14 PFLOP/s, 58% of the bf16 rate that a large matrix product has; 1.50 ms under a
// cap, 3.1 under one past 64.  The MMAs alone take 0.82 ms as they are issued; with one
// role taken out (widening, softmax, MMAs) the whole is 10 to 20% less, with all three
// 0.32 ms; 62% of the issue slots, 23% of the exponentials' rate.
// 128-key steps with one S buffer take the same (their MMAs are quicker, N = 64 takes
// as long as N = 128, but a softmax waits for its S), and so do four warpgroups of
// softmax; one that takes weights before the maximum of the block is known, 20% more.
#include "kv_attention.cuh"

namespace moe {
namespace {

constexpr int kThreads = 640;             // two warpgroups of softmax, two that widen, one that issues and brings scales
constexpr int kWidenThreads = 256, kIssueWarp = 16;
constexpr int kLaunchRegs = 96;           // registers a thread at launch, split over the warpgroups
constexpr int kTileRows = 128;
constexpr int kKeys = 64;                 // keys per step of a tile
constexpr int kBlock = 128;               // keys widened at a time
constexpr int kStages = 2;                // of K and of V blocks
constexpr int kScaleSlots = 4;
constexpr uint32_t kTmemCols = 512;
// Rescaling O takes a step's time, so the reference begins kFirstHead below the maximum,
// from where it seldom has to move, and is put kHead below after kSettle steps, when a
// maximum seldom rises by much; until then there are 4096 keys at most, whose rounding to
// multiples of 2^-26 of the largest weight amounts to 2^-15.  (kHead from the start: 1006
// us for an 8192-token prompt instead of 968; never, which is not right for long contexts
// under a dominant key: 959.)
constexpr float kFirstHead = 2.0f;
constexpr int kSettle = 64;
// Registers by role (setmaxnreg); the launch refuses any other launch allocation.
constexpr int kRegsSoftmax = 136, kRegsWiden = 80, kRegsIssue = 48;
static_assert(256 * kRegsSoftmax + kWidenThreads * kRegsWiden + 128 * kRegsIssue <= kThreads * kLaunchRegs, "register split");

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;               // 64 dimensions = 128 bytes of a row each
  static constexpr int kTileBytes = kPanels * 128 * 128;
  static constexpr int kQ = 0;
  static constexpr int kV = 2 * kTileBytes;
  static constexpr int kK = kV + kStages * kTileBytes;
  static constexpr int kScale = kK + kStages * kTileBytes;          // [slot][8 groups of 16 keys] float4
  static constexpr int kBars = kScale + kScaleSlots * 8 * 16;
  static constexpr int kSmem = 1024 + kBars + 256;
  static constexpr uint32_t kTmemO = 256;              // S0, S1 (and P over them) at 0, 128; O0, O1 here
};

// mbarriers, in order.  S, P and O have one for each buffer of a tile, and each tile's
// issuing warp two for the blocks that it releases: two steps can be under way, and a
// barrier must neither count one warp's next arrival for another's missing one nor get
// two phases ahead of who waits for it.
enum { kQFull, kEmpty = kQFull + 2, kKFull = kEmpty + 4, kVFull = kKFull + 2, kSFull = kVFull + 2, kPFull = kSFull + 4,
       kOFull = kPFull + 4, kBarCount = kOFull + 4 };

// Instruction descriptor, kind::f16: D fp32, A and B f16, A K-major; B K-major or
// (mn) with its N dimension contiguous.
constexpr uint32_t idesc_f16(int N, bool mn) {
  return (1u << 4) | (mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
// Shared-memory matrix descriptors, 128-byte swizzle, as their low words (the high
// one is the same for all): Q and K have the contracted dimension contiguous; V, as
// the B operand of P V, its N dimension: 64-dimension blocks a panel apart (the
// leading offset), groups of 8 keys 1024 bytes (the stride offset, in both).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading) {
  return ((saddr & 0x3FFFFu) >> 4) | ((leading >> 4) << 16);
}
// By the lane with `lead`: the whole warp runs the issuing loop, so its control flow
// and addresses are uniform.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %6, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc),
      "r"(kDescHi), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %6, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc),
      "r"(kDescHi), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
      "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void tmem_st_x8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Waits for this thread's TMEM loads, x's among them: no use of x moves ahead of it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]),
                 "+r"(x[16]), "+r"(x[17]), "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]),
                 "+r"(x[23]), "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29]),
                 "+r"(x[30]), "+r"(x[31])::"memory");
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])::"memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// y, but -inf where x is (a select, not a branch).
__device__ __forceinline__ float keep_hidden(float x, float y) {
  float r;
  asm("{\n\t.reg .pred p;\n\tsetp.eq.f32 p, %1, 0fFF800000;\n\tselp.f32 %0, %1, %2, p;\n\t}" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
// capped_log2(x f, cap) + add of four scores of S.  The four reciprocals of 1 + exp(2y)
// are one reciprocal of their product, which stays below 2^121: from exp(2y) = 2^30 on,
// tanh is 1 to fp32.  f and cap_log2 are those of capped_log2, f times 2 log2(e).  (A
// reciprocal for each score: 90 us for the windowed prompts instead of 84, 1704 for an
// 8192-token prompt under a cap instead of 1503.)
__device__ __forceinline__ void capped4(const uint32_t* x, float f, float cap_log2, float add, float* y) {
  float a[4];
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    float z0, z1;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), f2_pack(f, f)), z0, z1);
    asm("min.NaN.f32 %0, %1, 0f41F00000;" : "=f"(z0) : "f"(z0));
    asm("min.NaN.f32 %0, %1, 0f41F00000;" : "=f"(z1) : "f"(z1));
    f2_unpack(f2_add(f2_pack(ex2(z0), ex2(z1)), f2_pack(1.0f, 1.0f)), a[e], a[e + 1]);
  }
  const float p01 = a[0] * a[1], p23 = a[2] * a[3];
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(p01 * p23));
  const float r01 = r * p23, r23 = r * p01;
  const uint64_t m = f2_pack(-2.0f * cap_log2, -2.0f * cap_log2), c = f2_pack(cap_log2 + add, cap_log2 + add);
  f2_unpack(f2_fma(f2_pack(r01 * a[1], r01 * a[0]), m, c), y[0], y[1]);
  f2_unpack(f2_fma(f2_pack(r23 * a[3], r23 * a[2]), m, c), y[2], y[3]);
}
// 16 bytes read once by this CTA (no place in L1, what shared memory leaves of
// it), or zeros without a read; no branch either way.
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p, bool on) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"(static_cast<uint32_t>(on)));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds16f(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The largest |x| of 8 elements; NaN if one is.
template <bool F16>
__device__ __forceinline__ float abs_max8(const uint4& u) {
  uint32_t m;
  if constexpr (F16) {
    const auto h = [](uint32_t x) { return *reinterpret_cast<const __half2*>(&x); };
    const __half2 r = __hmax2_nan(__hmax2_nan(__habs2(h(u.x)), __habs2(h(u.y))), __hmax2_nan(__habs2(h(u.z)), __habs2(h(u.w))));
    m = *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const auto h = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    const __nv_bfloat162 r = __hmax2_nan(__hmax2_nan(__habs2(h(u.x)), __habs2(h(u.y))), __hmax2_nan(__habs2(h(u.z)), __habs2(h(u.w))));
    m = *reinterpret_cast<const uint32_t*>(&r);
  }
  const float2 f = pair_to_float<F16>(m);
  return fmax_nan(f.x, f.y);
}

// Steps [first, end) of kKeys keys that the rows [r0, r1) of a sequence see.
struct Steps {
  int first, end;
};
__device__ __forceinline__ Steps steps_of(const AttnArgs& a, const Seq& s, int r0, int r1) {
  return {first_key(a.d, s, r0 / a.G) / kKeys, (end_key(a.d, s, (r1 - 1) / a.G) + kKeys - 1) / kKeys};
}

// A bounded wait in little code (there are many of them, and the loops around them have
// to stay in the instruction caches): gives up after kWaitClocks, a second or so, or
// when another role has.
constexpr long long kWaitClocks = 2000000000ll;
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort || clock64() - t0 > kWaitClocks) {
      *abort = 1;
      set_err(err, MOE_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}

// A unit: up to 256 rows of a sequence.  Units of sequence b start at cu[b] * G / 256 +
// min(b, cu[b] * G / 33): enough for its rows whatever cu is if it has more than 32, as
// both terms of the minimum then grow by one at least, and nothing has to be summed; those
// with fewer, or none, add next to no units.  A unit's keys are cut into `splits` runs of
// `chunk` steps (an even number: whole blocks), fewer than asked for where they would be
// short.
__host__ __device__ __forceinline__ uint32_t units_before(uint32_t b, uint32_t rows) {
  const uint32_t many = rows / (kDecodeRows + 1);
  return rows / (2 * kTileRows) + (many < b ? many : b);
}
struct Unit {
  int b, rows, row0, row_end, splits, chunk;
  Seq s;
  Steps all;
};
constexpr int kMinChunk = 8;             // steps
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, int unit, int splits) {
  const moe_kv_cache& kc = a.d.cache;
  const auto unit0 = [&](int b) {
    return static_cast<int>(units_before(b, static_cast<uint32_t>(__ldg(kc.cu_new + b)) * a.G));   // at most 2^30 rows
  };
  Unit u;
  u.splits = 0;
  u.b = warp_find(kc.batch, unit, unit0);
  int32_t bad = 0;
  u.s = load_seq(a.d, u.b, &bad);          // faults are told by the decode kernel
  u.rows = u.s.n * a.G;
  if (u.rows <= kDecodeRows) return u;
  const int tiles2 = (u.rows + 2 * kTileRows - 1) / (2 * kTileRows);
  const int nth = tiles2 - 1 - (unit - unit0(u.b));         // the last rows, with the most keys, first
  if (nth < 0 || nth >= tiles2) return u;
  u.row0 = nth * 2 * kTileRows;
  u.row_end = min(u.rows, u.row0 + 2 * kTileRows);
  u.all = steps_of(a, u.s, u.row0, u.row_end);
  const int steps = u.all.end - u.all.first;
  u.chunk = steps;
  if (splits > 1) {
    u.all.first &= ~1;
    u.chunk = max(kMinChunk, ((u.all.end - u.all.first + splits - 1) / splits + 1) & ~1);
  }
  u.splits = (u.all.end - u.all.first + u.chunk - 1) / u.chunk;
  return u;
}
// A split's part: m[256], l[256], O[256][D], O not divided by l.
template <int D>
constexpr int64_t kSplitFloats = 2 * kTileRows * (D + 2);

// Caps: none; up to kCapDirect, on the way to the weights; past it, by bending S first.
enum Cap { kNoCap, kCap, kBend };
template <bool F16, int D, Cap MODE>
__device__ __forceinline__ void prefill(const AttnArgs& a, int splits) {
  constexpr bool CAP = MODE == kCap;
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_nan;
  const moe_kv_attention_desc& d = a.d;
  const moe_kv_cache& kc = d.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2;
  const int H = kc.kv_heads, P = kc.page_size, page_shift = 31 - __clz(P);

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::kBars;
  const auto bar = [&](int i) { return bars + 8 * i; };
  if (tid == 0) {
    for (int i = 0; i < kBarCount; ++i) {
      const bool rows128 = i < kQFull + 2 || (i >= kPFull && i < kPFull + 4);
      const int widen = i >= kKFull && i < kVFull ? kWidenThreads + 1 : i >= kVFull && i < kVFull + 2 ? kWidenThreads : 0;
      mbar_init(bar(i), widen ? widen : rows128 ? 128 : 1);
    }
    s_abort = 0;
    s_nan = 0;
    fence_barrier_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int split = blockIdx.x % splits, h = blockIdx.x / splits % H;
  const Unit w = unit_of(a, blockIdx.x / splits / H, splits);
  if (split >= w.splits) return;           // the unit has no rows, or needs fewer splits
  // (not before the wait above: a CTA of the kernel before this one may still want TMEM)
  if (warp == kIssueWarp) {
    tmem_alloc(smem_u32(&s_tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int b = w.b, rows = w.rows, row0 = w.row0, row_end = w.row_end;
  const Seq s = w.s;
  const int tiles = row_end - row0 > kTileRows ? 2 : 1;
  // this CTA's steps, of all rows and of each tile's (a tile may have none in a split)
  const Steps all = {w.all.first + split * w.chunk, min(w.all.end, w.all.first + (split + 1) * w.chunk)};
  const auto mine = [&](int r0, int r1) {
    const Steps m = steps_of(a, s, r0, r1);
    return Steps{max(m.first, all.first), min(m.end, all.end)};
  };
  const Steps mine0 = mine(row0, min(row0 + kTileRows, row_end));
  const Steps mine1 = tiles == 2 ? mine(row0 + kTileRows, row_end) : Steps{all.end, all.end};
  const int block0 = all.first >> 1, block1 = (all.end + 1) >> 1;   // blocks to widen

  // A warp of the issuing role goes on or gives up as one.  The other roles go on with
  // their loops when a lane has given up (every later wait ends at once then), so that no
  // lane leaves its warp, and look at s_abort in the end.
  const auto wait_lane = [&](int i, int phase) { return wait_for(bar(i), phase & 1, &s_abort, d.err); };
  const auto wait = [&](int i, int phase) { return static_cast<bool>(__all_sync(0xffffffffu, wait_lane(i, phase))); };

  if (wg == 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    const int i = warp - kIssueWarp;
    if (i < tiles) {
      // ------------------------------------------------------------ MMA issue, a warp for each tile
      // S has two buffers a tile: step g + 2 goes where step g was.  Per step: P V of
      // step g, then S of step g + 2 over the space that its P took (MMAs of one thread
      // run in order), so that S of step g + 1 is there when its softmax begins.  The
      // commit of S tells of that P V too; the last two steps, which have no S after
      // them, have a commit of their own.  Every block is waited for and released by
      // both warps, whether its tile reads it or not.
      const uint32_t id_s = idesc_f16(kKeys, false), id_o = idesc_f16(D, true);
      const uint32_t lead = elect_one();
      const Steps m = i ? mine1 : mine0;
      const uint32_t to = tmem + C::kTmemO + i * D, ts = tmem + i * 128;
      const uint32_t qd = desc_lo(sbase + C::kQ + i * C::kTileBytes, 16);
      bool ok = wait(kQFull + i, 0), any = false;
#pragma unroll 1
      for (int g2 = (all.first & ~1) - 2; ok && g2 < all.end; g2 += 2) {
        const int vb = (g2 >> 1) - block0, kb = vb + 1;               // blocks that are read (V of -1: none)
        const bool more = kb < block1 - block0;
        if (vb >= 0) ok = wait(kVFull + (vb & 1), vb >> 1);
        if (ok && more) ok = wait(kKFull + (kb & 1), kb >> 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int buf = 0; buf < 2; ++buf) {
          const int g = g2 + buf;
          const uint32_t half = buf * kKeys;
          const bool next = g + 2 >= m.first && g + 2 < m.end;
          if (g >= m.first && g < m.end) {
            ok = wait(kPFull + 2 * i + buf, (g - m.first) >> 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t vd = desc_lo(sbase + C::kV + (vb & 1) * C::kTileBytes + half * 128, 16384);
            const uint32_t acc = g > m.first;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k) mma_ts(to, ts + half + 8 * k, vd + 128 * k, id_o, k > 0 ? 1u : acc, lead);
            if (!next) commit(bar(kOFull + 2 * i + buf), lead);
          }
          if (next) {
            const uint32_t kd = desc_lo(sbase + C::kK + (kb & 1) * C::kTileBytes + half * 128, 16);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t at = (k >> 2) * 1024 + (k & 3) * 2;
              mma_ss(ts + half, qd + at, kd + at, id_s, k > 0 ? 1u : 0u, lead);
            }
            commit(bar(kSFull + 2 * i + buf), lead);
            any = true;
          }
        }
        if (ok) commit(bar(kEmpty + 2 * i + (kb & 1)), lead);
      }
      if (!ok && any && lead) {
        // the MMAs in flight end before TMEM is freed: the commit below follows them
        int dummy = 0;
        umma_commit(bar(kQFull + i));    // completes phase 1 of a barrier that nobody else waits on any more
        for (int k = 1; k < 128; ++k) mbar_arrive(bar(kQFull + i));
        mbar_wait_bounded(bar(kQFull + i), 1, &dummy, nullptr, kWaitLimitNs / 10);
      }
      __syncwarp();
    } else if (i == 2) {
      // ------------------------------------------------------------ scales, a lane for each 16-key group
      // of a block: K's, and V's as its logarithm and inverse, which is what the weights
      // take.  Then, of each step's four groups: the size of its largest V scale (its
      // exponent, not below 2^-60 of the largest of all), and in place of the first one's
      // NaN where that is a new one, else how far a maximum may lead the reference.
      const auto page_of = [&](int j) {
        const int key = j * kBlock + lane * 16;
        return lane < 8 && key < s.len ? __ldg(kc.page_table + b * kc.table_ld + (key >> page_shift)) : -1;
      };
      const auto scales_of = [&](int page) {             // 0 where there are no keys
        if (page < 0 || page >= kc.pages) return make_float2(0.0f, 0.0f);
        const int64_t at = static_cast<int64_t>(page) * H + h;
        return make_float2(__ldg(kc.k_scale + at), __ldg(kc.v_scale + at));
      };
      float2 next = scales_of(page_of(block0));
      int page = page_of(block0 + 1), size = 0, largest = 0;
#pragma unroll 1
      for (int j = block0; j < block1; ++j) {
        const int n = j - block0;
        const float2 now = next;
        next = scales_of(page);                          // under way during the wait
        page = page_of(j + 2);
        const float v = fmaxf(now.y, kMinScale);
        int most = now.y > 0.0f ? __float_as_int(v) >> 23 : 0;
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        float w = kLazy;
#pragma unroll
        for (int step = 0; step < 2; ++step) {
          const int of = __shfl_sync(0xffffffffu, most, 4 * step);
          const bool other = of != 0 && abs(of - size) > kNear;
          if (other) {
            largest = max(largest, of);
            size = max(of, largest - 60);
          }
          if (lane >> 2 == step) w = lane & 3 ? static_cast<float>(size) : other ? __uint_as_float(0x7FC00000u) : kLazy;
        }
        // a tile's e-th release: V up to block e - 1 is read, so the weights of that are done
        if (n >= 2) {
          wait_lane(kEmpty + (n & 1), (n - 2) >> 1);
          if (tiles == 2) wait_lane(kEmpty + 2 + (n & 1), (n - 2) >> 1);
        }
        if (lane < 8)
          *reinterpret_cast<float4*>(smem + C::kScale + ((n & (kScaleSlots - 1)) * 8 + lane) * 16) =
              make_float4(now.x, __log2f(v), __fdividef(1.0f, v), w);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kKFull + (n & 1)));
      }
    }
  } else if (wg >= 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWiden));
    // ------------------------------------------------------------ widening of K and V
    constexpr int kRowsPer = kWidenThreads / (D / 16);  // rows the two warpgroups take at a time
    constexpr int kIter = kBlock / kRowsPer;
    // four lanes take half a 128-byte row of codes, the next four that of the next row:
    // their stores then fall on all banks, whatever the swizzle
    const int t = tid - 256, panel = (t >> 5) & (C::kPanels - 1);
    const int r0 = ((t >> 2) & 7) | (t >> (C::kPanels == 2 ? 6 : 5)) << 3, ch = panel * 4 + (t & 3);
    const int hi_all = end_key(d, s, row0 / a.G), lo_all = first_key(d, s, (row_end - 1) / a.G);
    // page of 16-key group pages_from + lane (whole blocks: 32 groups from a multiple
    // of 8), and of the 32 groups after those
    int pages_from = block0 * 8, pages, pages_next;
    bool bad_page = false;
    const auto look_up = [&](int from) {
      const int key = (from + lane) << 4;
      int page = key < s.len ? __ldg(kc.page_table + b * kc.table_ld + (key >> page_shift)) : 0;
      if (page < 0 || page >= kc.pages) {
        bad_page = true;
        page = -1;
      }
      return page;
    };
    pages = look_up(pages_from);
    pages_next = look_up(pages_from + 32);
    uint4 reg[2][kIter];                               // K's and V's codes, loaded a block ahead
    // Address of a 16-key group's rows: a 32 x 32 bit product for the page (strides are
    // multiples of 16), a term for the group that all lanes share and one for the lane.
    // The row within its page is (i, j)'s part plus r0's, whatever the page size.
    const auto load = [&](uint4& r, int i, int j, const uint8_t* base, uint32_t page_ld16, int64_t slot_ld) {
      const int key0 = j * kBlock + i * kRowsPer;
      const int page = __shfl_sync(0xffffffffu, pages, ((key0 + r0) >> 4) - pages_from);
      const uint8_t* p = base + (static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_ld16 << 4) + (key0 & (P - 1)) * slot_ld;
      // past the end, or a page that is none: zeros
      r = ldg_stream(p, key0 + r0 < s.len && page >= 0);
    };
    const uint8_t* base[2] = {kc.k + h * kc.k_head_ld + (r0 & (P - 1)) * kc.k_slot_ld + ch * 16,
                              kc.v + h * kc.v_head_ld + (r0 & (P - 1)) * kc.v_slot_ld + ch * 16};
    const uint32_t page_ld16[2] = {static_cast<uint32_t>(kc.k_page_ld >> 4), static_cast<uint32_t>(kc.v_page_ld >> 4)};
#pragma unroll
    for (int i = 0; i < kIter; ++i) load(reg[0][i], i, block0, base[0], page_ld16[0], kc.k_slot_ld);
#pragma unroll
    for (int i = 0; i < kIter; ++i) load(reg[1][i], i, block0, base[1], page_ld16[1], kc.v_slot_ld);
#pragma unroll 1
    for (int j = block0; j < block1; ++j) {
      const int n = j - block0, st = n & 1;
      const bool more = j + 1 < block1;
      if (more) {
        if ((j + 1) * 8 - pages_from == 32) {
          pages_from += 32;
          pages = pages_next;
          pages_next = look_up(pages_from + 32);
        }
      }
#pragma unroll
      for (int is_v = 0; is_v < 2; ++is_v) {
        // A tile's e-th release: K up to block e and V up to block e - 1 are read.  V of block
        // n takes the place of n - 2's; K of block n + 1, which comes next, that of n - 1's.
        if (is_v && n > 0) {
          wait_lane(kEmpty + ((n - 1) & 1), (n - 1) >> 1);
          if (tiles == 2) wait_lane(kEmpty + 2 + ((n - 1) & 1), (n - 1) >> 1);
        }
        if (is_v && (j * kBlock < lo_all || (j + 1) * kBlock > hi_all)) {
          // A NaN must not meet the zero weight of a row that does not see it (as in the
          // decode kernel): blocks with such rows lose theirs here, and the rows that do
          // see them get them in the end.
          uint32_t any = 0;
#pragma unroll
          for (int i = 0; i < kIter; ++i) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&reg[is_v][i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t bad = nan_codes(w[k]);
              any |= bad;
              w[k] &= ~((bad >> 7) * 0xFFu);
            }
          }
          if (any) s_nan = 1;
        }
        const uint32_t row = sbase + (is_v ? C::kV : C::kK) + st * C::kTileBytes + panel * 16384 + r0 * 128;
        const uint32_t at_lo = row + (((2 * (t & 3)) ^ (r0 & 7)) << 4), at_hi = row + (((2 * (t & 3) + 1) ^ (r0 & 7)) << 4);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const uint4 w = reg[is_v][i];
          if (more)
            load(reg[is_v][i], i, j + 1, base[is_v], page_ld16[is_v], is_v ? kc.v_slot_ld : kc.k_slot_ld);
          sts16(at_lo + i * kRowsPer * 128,
                make_uint4(e4m3x2_to_f16x2(w.x & 0xFFFF), e4m3x2_to_f16x2(w.x >> 16), e4m3x2_to_f16x2(w.y & 0xFFFF),
                           e4m3x2_to_f16x2(w.y >> 16)));
          sts16(at_hi + i * kRowsPer * 128,
                make_uint4(e4m3x2_to_f16x2(w.z & 0xFFFF), e4m3x2_to_f16x2(w.z >> 16), e4m3x2_to_f16x2(w.w & 0xFFFF),
                           e4m3x2_to_f16x2(w.w >> 16)));
        }
        fence_proxy_async_shared();
        mbar_arrive(bar((is_v ? kVFull : kKFull) + st));
      }
    }
    if (bad_page) set_err(d.err, MOE_DEV_BAD_INDEX);
  } else if (wg < tiles) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------ softmax and output of tile wg
    const int t = tid & 127;
    const int r = row0 + wg * kTileRows + t;
    const bool live = r < rows;
    const int i = min(r, rows - 1) / a.G, head = h * a.G + min(r, rows - 1) - i * a.G;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;       // this warp's TMEM lanes (bits 16 and up)
    const uint32_t ts = tmem + lanes + wg * 128, to = tmem + lanes + C::kTmemO + wg * D;
    float qs = 0.0f;
    {
      // Each warp brings its 32 rows in, kLanes lanes to a row, all loads in flight at once.
      constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
      uint4 w[kLanes];
      const int sub = lane / kLanes, c16 = lane % kLanes;              // row of a group, 16-byte chunk of the row
      const int first = row0 + wg * kTileRows + (warp & 3) * 32;
      // (token, head) of each row: one division, and then small ones by a reciprocal
      // ((x + 1/2) / G in fp32 has the right whole part for x < G + 32 < 2^17)
      const int i0 = min(first, rows - 1) / a.G, g0 = min(first, rows - 1) - i0 * a.G;
      const float inv_g = 1.0f / static_cast<float>(a.G);
#pragma unroll
      for (int k = 0; k < kLanes; ++k) {
        const int x = min(g0 + k * kAtOnce + sub, g0 + max(rows - 1 - first, 0));
        const int up = static_cast<int>((static_cast<float>(x) + 0.5f) * inv_g);
        w[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(d.q) + (s.c0 + i0 + up) * d.q_token_ld +
                                                    (h * a.G + x - up * a.G) * d.q_head_ld) + c16);
      }
      // The rows' maxima: of each lane's 8 elements, then over a row's lanes for all rows
      // at once -- halves of the rows change sides at every step, until a lane has one row.
      float amax[kLanes];
#pragma unroll
      for (int k = 0; k < kLanes; ++k) amax[k] = abs_max8<F16>(w[k]);
#pragma unroll
      for (int half = kLanes / 2; half > 0; half >>= 1)
#pragma unroll
        for (int k = 0; k < half; ++k) {
          const bool up = (c16 & half) != 0;
          const float give = up ? amax[k] : amax[k + half], keep = up ? amax[k + half] : amax[k];
          const float got = __shfl_xor_sync(0xffffffffu, give, half);
          amax[k] = fmax_nan(keep, got);
        }
      float mul, inv;
      row_scale(amax[0], mul, inv);        // of row c16 * kAtOnce + sub
      mul = copysignf(mul, d.sm_scale);
      // this thread's own row is row lane of the 32
      qs = __shfl_sync(0xffffffffu, inv, lane % kAtOnce * kLanes + lane / kAtOnce);
      const uint32_t tile = sbase + C::kQ + wg * C::kTileBytes + (c16 >> 3) * 16384;
#pragma unroll
      for (int k = 0; k < kLanes; ++k) {
        float f[8];
        unpack8<F16>(w[k], f);
        const float m = __shfl_sync(0xffffffffu, mul, sub * kLanes + k);
        const int row = (warp & 3) * 32 + k * kAtOnce + sub;           // of the tile
        sts16(tile + row * 128 + (((c16 & 7) ^ (row & 7)) << 4),
              make_uint4(f16x2(f[0] * m, f[1] * m), f16x2(f[2] * m, f[3] * m), f16x2(f[4] * m, f[5] * m),
                         f16x2(f[6] * m, f[7] * m)));
      }
      qs *= fabsf(CAP ? d.sm_scale / d.softcap : d.sm_scale * kLog2e);
      fence_proxy_async_shared();
      mbar_arrive(bar(kQFull + wg));
    }
    // What a row's S takes to be a score, of the keys with this scale.  -inf, which stands
    // for a key that is not seen, must not meet a zero; scores so small are 0 anyway.
    const auto factor = [&](float k_scale) { return fmax_nan(qs * k_scale, FLT_MIN); };
    const auto score = [&](float x, float f, float add) {
      if constexpr (CAP) return keep_hidden(x, capped_log2(x * f, d.softcap * kLog2e) + add);
      return fmaf(x, f, add);
    };
    const int lo = first_key(d, s, i), hi = end_key(d, s, i);
    const int tile_r1 = min(rows, row0 + (wg + 1) * kTileRows) - 1;
    const int lo_last = first_key(d, s, tile_r1 / a.G), hi_first = end_key(d, s, (row0 + wg * kTileRows) / a.G);
    const Steps m = wg ? mine1 : mine0;
    // running reference (ref: the same, 0 while -inf), sum, and the largest score so far
    float top = -INFINITY, ref = 0.0f, sum = 0.0f, peak = -INFINITY;
    float size = 0.0f;                                   // of the V scales that it goes with
#pragma unroll 1
    for (int g = m.first; g < m.end; ++g) {
      const int n = g - m.first, buf = g & 1;
      wait_lane(kSFull + 2 * wg + buf, n >> 1);
      tc_fence_after();
      const uint32_t at = ts + buf * kKeys;
      const uint32_t scale = sbase + C::kScale + (((g >> 1) - block0) & (kScaleSlots - 1)) * 128 + buf * 64;
      if constexpr (MODE == kBend) {
        // S as if the score had been capped, x tanh(y) / y, in its place
        const float bend = 1.0f / (d.softcap * kLog2e);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t x[16];
          tmem_ld_32x32b_x16(at + 16 * k, x);
          tmem_ld_wait_for(x);
          const float f = factor(lds16f(scale + k * 16).x) * bend;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[e] = __float_as_uint(__uint_as_float(x[e]) * tanh_ratio(__uint_as_float(x[e]) * f));
          tmem_st_x16(at + 16 * k, x);
        }
        tmem_st_wait();
      }
      uint32_t x[2][32];
      tmem_ld_32x32b_x32(at, x[0]);
      tmem_ld_32x32b_x32(at + 32, x[1]);
      const bool edge = g * kKeys < lo_last || (g + 1) * kKeys > hi_first;
      tmem_ld_wait_for(x[0]);
      tmem_ld_wait_for(x[1]);
      if (edge) {                          // one branch, not one for each element
        const uint32_t from = lo - g * kKeys, seen = hi - lo;
#pragma unroll
        for (uint32_t e = 0; e < kKeys; ++e)
          if (e - from >= seen) x[e >> 5][e & 31] = 0xFF800000u;
      }
      // A score is a function of S that does not fall within a group of one scale (q has
      // taken sm_scale's sign), so the maximum needs it once for each group.
      float best = -INFINITY, factors[4], lead = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t* y = &x[k >> 1][(k & 1) * 16];
        float top16 = __uint_as_float(y[0]);
#pragma unroll
        for (int e = 1; e < 15; e += 2)
          top16 = fmaxf(fmaxf(top16, __uint_as_float(y[e])), __uint_as_float(y[e + 1]));
        top16 = fmaxf(top16, __uint_as_float(y[15]));
        const float4 sc = lds16f(scale + k * 16);
        factors[k] = factor(sc.x);
        if (k == 0) lead = sc.w;
        best = fmaxf(best, score(top16, factors[k], sc.y));
      }
      if (__any_sync(0xffffffffu, !(best <= top + lead) || n == kSettle)) {
        // The reference goes with the size of the V scales, down as well as up, so that weights
        // are as precise as before (fp32 holds what there is), and then with the maximum.
        const float now = lds16f(scale + 16).w, base = top + (now - size);
        peak += now - size;
        size = now;
        float next = base;
        if (best > base + kLazy || n == kSettle) next = fmaxf(peak, best) - (n >= kSettle ? kHead : kFirstHead);
        const float keep = next == -INFINITY ? 1.0f : ex2(top - next);
        top = next;
        ref = next == -INFINITY ? 0.0f : next;
        sum *= keep;
        if (n > 0) {
          // P V of the step before is in: by the commit of S of the step after, if there is one
          const bool last = g + 1 == m.end;
          wait_lane((last ? kOFull : kSFull) + 2 * wg + (buf ^ 1), last ? 0 : (n + 1) >> 1);
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(to + 16 * k, o);
            tmem_ld_wait_for(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
            tmem_st_x16(to + 16 * k, o);
          }
        }
      }
      peak = fmaxf(peak, best);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t p[8];
        const float4 sc = lds16f(scale + k * 16);
        const float f = factors[k], v = sc.y - ref;
        const uint64_t f2 = f2_pack(f, f), v2 = f2_pack(v, v);
        uint64_t acc[2] = {0, 0};
        const uint32_t* xk = &x[k >> 1][(k & 1) * 16];
        float y[16];
        if constexpr (CAP) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) capped4(xk + e, 2.0f * kLog2e * f, d.softcap * kLog2e, v, y + e);
          if (edge) {
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = keep_hidden(__uint_as_float(xk[e]), y[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            f2_unpack(f2_fma(f2_pack(__uint_as_float(xk[e]), __uint_as_float(xk[e + 1])), f2, v2), y[e], y[e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          y[e] = ex2(y[e]);
          y[e + 1] = ex2(y[e + 1]);
          acc[(e >> 1) & 1] = f2_add(acc[(e >> 1) & 1], f2_pack(y[e], y[e + 1]));
          p[e / 2] = f16x2(y[e], y[e + 1]);
        }
        float a0, a1;
        f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
        sum = fmaf(a0 + a1, sc.z, sum);
        tmem_st_x8(at + 8 * k, p);                       // over S, which is in registers
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(kPFull + 2 * wg + buf));
    }
    const bool none = m.first >= m.end;                  // of this split's keys; O was never written then
    if (!none) wait_lane(kOFull + 2 * wg + ((m.end - 1) & 1), 0);
    if (__all_sync(0xffffffffu, *static_cast<volatile int*>(&s_abort) == 0)) {
      tc_fence_after();
      const float inv = none ? 0.0f : w.splits > 1 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      // Output rows go through shared memory, where Q was (no MMA is left to read it), so
      // that a store takes whole rows and not 16 bytes of each of 32 (8192-token prompt 972
      // -> 960 us); in short loops, as their code is fetched for a single use.
      const uint32_t stage = sbase + C::kQ + wg * C::kTileBytes + (warp & 3) * (32 * 2 * D), own = stage + lane * (2 * D);
      float* part = a.parts + static_cast<int64_t>(blockIdx.x) * kSplitFloats<D> + wg * kTileRows + t;
      if (w.splits > 1 && live) {
        part[0] = top;
        part[2 * kTileRows] = sum;
      }
      part += 4 * kTileRows + (wg * kTileRows + t) * (D - 1);
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(to + 32 * k, o);
        tmem_ld_wait_for(o);
        float f[4][8];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e >> 3][e & 7] = none ? 0.0f : __uint_as_float(o[e]) * inv;
        if (w.splits == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sts16(own + (((4 * k + e) ^ (lane & 7)) << 4), pack8<F16>(f[e]));
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float* x = &f[e >> 1][(e & 1) * 4];
            reinterpret_cast<float4*>(part)[8 * k + e] = make_float4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      if (live && *static_cast<volatile int*>(&s_nan)) {
        // NaN codes that were taken out of blocks with rows that do not see them all
        const int hi_all = end_key(d, s, row0 / a.G), lo_all = first_key(d, s, (row_end - 1) / a.G);
        const int to_key = min(hi, all.end * kKeys);
        for (int key = max(lo, all.first * kKeys); key < to_key; ++key) {
          const int k0 = key & ~(kBlock - 1);
          if (!(k0 < lo_all || k0 + kBlock > hi_all)) {
            key = max(key, (hi_all & ~(kBlock - 1)) - 1);
            continue;
          }
          const int page = __ldg(kc.page_table + b * kc.table_ld + (key >> page_shift));
          if (page < 0 || page >= kc.pages) continue;
          const uint8_t* vp = kc.v + page * kc.v_page_ld + h * kc.v_head_ld + (key & (P - 1)) * kc.v_slot_ld;
#pragma unroll 1
          for (int e = 0; e < D; ++e) {
            if ((vp[e] & 0x7F) != 0x7F) continue;
            if (w.splits == 1) {
              const uint32_t at = own + (((e >> 3) ^ (lane & 7)) << 4) + 2 * (e & 7);
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(0x7FFF)) : "memory");   // of either type
            } else {
              part[e] = __uint_as_float(0x7FC00000u);
            }
          }
        }
      }
      if (w.splits == 1) {
        __syncwarp();
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;           // as Q was read
        const int sub = lane / kLanes, c16 = lane % kLanes, first = row0 + wg * kTileRows + (warp & 3) * 32;
        const int i0 = first / a.G, g0 = first - i0 * a.G;
        const float inv_g = 1.0f / static_cast<float>(a.G);
        uint16_t* op = static_cast<uint16_t*>(d.out) + (s.c0 + i0) * d.o_token_ld + h * a.G * d.o_head_ld + c16 * 8;
#pragma unroll 4
        for (int local = sub; local < 32; local += kAtOnce) {
          const int x = g0 + local, up = static_cast<int>((static_cast<float>(x) + 0.5f) * inv_g);
          const uint4 v = lds16(stage + local * (2 * D) + ((c16 ^ (local & 7)) << 4));
          if (first + local < rows)
            *reinterpret_cast<uint4*>(op + up * d.o_token_ld + (x - up * a.G) * d.o_head_ld) = v;
        }
      }
      if (live && w.splits == 1 && d.lse != nullptr)
        d.lse[static_cast<int64_t>(s.c0 + i) * d.q_heads + head] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool F16, int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(const __grid_constant__ AttnArgs a, int splits) {
  prefill<F16, D, CAP ? kCap : kNoCap>(a, splits);
}
// A kernel of its own: as a branch of the two above its code alone costs their calls up
// to 7% (windowed prompts under a cap 84 -> 90 us, chunks 573 -> 584).
template <bool F16, int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_bend_kernel(const __grid_constant__ AttnArgs a, int splits) {
  prefill<F16, D, kBend>(a, splits);
}

// Fewer units than SMs: their keys are split so that every SM has some, if they are
// long enough for it (what the page table can hold is all the host knows of them).
int prefill_splits(const AttnArgs& a, int64_t units) {
  const int64_t keys = static_cast<int64_t>(a.d.cache.max_pages) * a.d.cache.page_size;
  const int64_t by_sms = num_sms() / units, by_keys = keys / (kMinChunk * kKeys);
  const int64_t n = by_sms < by_keys ? by_sms : by_keys;
  return n < 1 ? 1 : static_cast<int>(n);
}

// Joins the splits' parts, a warp to a row, in the order of the keys.
constexpr int kJoinRows = 8;             // rows (warps) of a CTA
template <bool F16, int D>
__global__ void __launch_bounds__(32 * kJoinRows) kv_prefill_join_kernel(const __grid_constant__ AttnArgs a, int splits) {
  const moe_kv_attention_desc& d = a.d;
  const int H = d.cache.kv_heads, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kPer = 2 * kTileRows / kJoinRows;
  const int at = blockIdx.x / kPer, h = at % H;
  const Unit w = unit_of(a, at / H, splits);
  const int local = blockIdx.x % kPer * kJoinRows + (threadIdx.x >> 5);
  if (w.splits <= 1 || w.row0 + local >= w.row_end) return;
  const float* part = a.parts + static_cast<int64_t>(at) * splits * kSplitFloats<D>;
  float top = -INFINITY;
  for (int k = lane; k < w.splits; k += 32) top = fmaxf(top, __ldcg(part + k * kSplitFloats<D> + local));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  constexpr int E = D / 32;
  float acc[E], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 8
  for (int k = 0; k < w.splits; ++k) {
    const float* p = part + k * kSplitFloats<D>;
    const float pm = __ldcg(p + local), pl = __ldcg(p + 2 * kTileRows + local);
    const float keep = pm == -INFINITY ? 1.0f : ex2(pm - top);   // a part without weights may hold a NaN
    sum = fmaf(pl, keep, sum);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(p + 4 * kTileRows + static_cast<int64_t>(local) * D + lane * E + e));
      acc[e] = fmaf(v.x, keep, acc[e]);
      acc[e + 1] = fmaf(v.y, keep, acc[e + 1]);
    }
  }
  const int r = w.row0 + local, i = r / a.G, head = h * a.G + r - i * a.G;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* op = static_cast<uint16_t*>(d.out) + (w.s.c0 + i) * d.o_token_ld + head * d.o_head_ld + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(op + e) = pair_from_float<F16>(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && d.lse != nullptr)
    d.lse[static_cast<int64_t>(w.s.c0 + i) * d.q_heads + head] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

template <bool F16, int D, Cap MODE>
int launch(const AttnArgs& a, cudaStream_t st) {
  static int prepared[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  void (*kernel)(AttnArgs, int);
  if constexpr (MODE == kBend) kernel = kv_prefill_bend_kernel<F16, D>;
  else kernel = kv_prefill_kernel<F16, D, MODE == kCap>;
  if (!__atomic_load_n(&prepared[dev], __ATOMIC_ACQUIRE)) {
    // the register split counts on exactly the launch allocation
    cudaFuncAttributes attr;
    MOE_CUDA_TRY(cudaFuncGetAttributes(&attr, kernel));
    if (attr.numRegs != kLaunchRegs) return MOE_ERR_UNSUPPORTED;
    MOE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem));
    __atomic_store_n(&prepared[dev], 1, __ATOMIC_RELEASE);
  }
  const int64_t units = static_cast<int64_t>(units_before(a.d.cache.batch, static_cast<uint32_t>(a.d.T * a.G))) * a.d.cache.kv_heads;
  if (units == 0) return MOE_OK;           // max_q allows more rows than there are
  const int splits = prefill_splits(a, units);
  // (some 2^25 by the limits of the descriptor; with splits at most one for each SM)
  const dim3 grid(static_cast<unsigned>(units * splits));
  if (int rc = launch_pdl(kernel, grid, dim3(kThreads), Cfg<D>::kSmem, st, a, splits)) return rc;
  if (splits == 1) return MOE_OK;
  return launch_pdl(kv_prefill_join_kernel<F16, D>, dim3(static_cast<unsigned>(units * (2 * kTileRows / kJoinRows))),
                    dim3(32 * kJoinRows), 0, st, a, splits);
}

template <bool F16, int D>
int pick_cap(const AttnArgs& a, cudaStream_t st) {
  if (a.d.softcap > kCapDirect) return launch<F16, D, kBend>(a, st);
  return a.d.softcap > 0.0f ? launch<F16, D, kCap>(a, st) : launch<F16, D, kNoCap>(a, st);
}

}  // namespace

size_t kv_prefill_workspace() { return static_cast<size_t>(num_sms()) * kSplitFloats<128> * sizeof(float); }

int kv_prefill_launch(const AttnArgs& a, cudaStream_t st) {
  const bool f16 = a.d.cache.dtype == MOE_DTYPE_F16;
  if (a.d.cache.dim == 64) return f16 ? pick_cap<true, 64>(a, st) : pick_cap<false, 64>(a, st);
  return f16 ? pick_cap<true, 128>(a, st) : pick_cap<false, 128>(a, st);
}

}  // namespace moe
