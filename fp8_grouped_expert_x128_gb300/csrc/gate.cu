// The router's logits: tokens times the gate's rows, fp32 sums (moe_gate).
//
//   logits[t, e] = sum_h x[t, h] * w[e, h]
//
// A skinny product: with few tokens it reads the gate (3.7 MB for 256 experts of
// hidden 7168) and should take as long as launching it; with many it reads the
// tokens, 256 multiply-adds a value, which is where GB300's tensor cores and its
// memory take equally long.  Up to 16 tokens are multiplied without the tensor cores, a
// CTA for one, two or four experts (gate_few_kernel).  More go through one kernel on the tensor cores
// (gate_kernel: tcgen05, 128 tokens by BN experts a CTA) whose tile and split follow
// their number:
//
//  * many tokens: BN = 256 in pairs of CTAs, so that a token's row is read once for 256
//    experts and a gate's row once for 256 tokens;
//  * fewer: the hidden dimension is split over a cluster of up to 8 CTAs, and then the
//    experts over narrower tiles, until there is a CTA for every SM.  The cluster
//    adds its parts through distributed shared memory, in the order of the ranks.
//
// Warp roles: one TMA producer (ring of stages of 64 columns, of 128 where BN is up to 128;
// 128-byte swizzle), one MMA issuer, and epilogue warps, four for every 64 experts.  Precision: the tensor
// cores cut what they add to a running sum, some 2^-24 of it a step, always towards
// zero; over 448 steps (hidden 7168) that is more than the logits of a router may be
// off.  So a sum runs over 512 columns only (32 steps; kRun), into one of two
// accumulators, and the epilogue warps add it in fp32, rounded to nearest, to sums in
// registers while the next 512 run.
//
// 16384 tokens of hidden 7168 by 256 experts take 50 us (5.1 TB/s, 1.2 PFLOP/s): bound by
// the copies into the SMs, and so are 256 (7.1 us), 512 (8.5), 1024 (10.8) and 2048 tokens (13.4)
// of it, whose narrower tiles bring each gate row into an SM once for every 128 tokens.  333 tokens
// of hidden 2040 by 60 take 4.1: launch, copies, a cluster barrier; one token by 256 2.0: launch and
// a round of loads.
#include <algorithm>

#include "gemm_common.cuh"
#include "kv_common.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;                     // tokens
constexpr int kCols = 64;                      // columns of a stage: 128 bytes, the swizzle's row
constexpr uint32_t kXBytes = kTile * kCols * 2;

constexpr int kMaxStages = 16;
constexpr int kRun = 4;                        // blocks of 128 columns that one accumulator sums

// BN experts a tile; kPair: two CTAs share the tile's gate rows and 256 tokens.
template <int BN, bool kPair>
struct Gate {
  static constexpr int kWRows = kPair ? BN / 2 : BN;         // gate rows that a CTA loads
  static constexpr int kSub = BN <= 128 ? 2 : 1;             // boxes of 64 columns in a stage
  static constexpr uint32_t kWBytes = kWRows * kCols * 2;    // of one box
  static constexpr int kEpi = BN > 64 ? BN / 16 : 4;         // epilogue warps
  static constexpr int kPer = BN > 64 ? 64 : BN;             // experts of a warp
  static constexpr int kLoad = BN >= 256 || BN < 32 ? 16 : 32;   // columns of one read of an accumulator (18 warps: 96 registers)
  static constexpr int kThreadCount = 64 + 32 * kEpi;
  static constexpr int kLd = BN + 4;                         // of the parts in shared memory, floats
  static constexpr uint32_t kTmem = 2 * BN;
};

struct GateArgs {
  float* logits;
  int64_t ld;
  int64_t T;
  int32_t* err;
  int32_t E, H, splits, n_tiles, box_rows, stages;
  uint64_t wait_limit_ns;
};

// kind::f16 with fp32 sums, both operands K-major, f16 or bf16.
__host__ __device__ constexpr uint32_t gate_idesc(bool f16, int M, int N) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool kPair>
__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kPair) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// A copy into this CTA whose barrier may be the even CTA's of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* map, uint32_t bar, int32_t x, int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// A barrier of the warps that know tensor memory (0 is all threads').
constexpr int kTmemBarrier = 1;
__device__ __forceinline__ void named_sync(int id, int threads) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void named_arrive(int id, int threads) { asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// A CTA's place: `rank` in its cluster of splits (x 2 in pairs) CTAs; in a pair the even
// CTA issues the MMAs of both (M = 256: its own 128 tokens and the odd one's), with half of
// the gate's rows in each one's shared memory.  The copies of both complete on the even
// one's barrier; commits arrive in both, the epilogue warps of both at the even one.
template <int BN, bool kPair, bool F16>
__global__ void __launch_bounds__(Gate<BN, kPair>::kThreadCount, 1)
    gate_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const GateArgs p) {
  using G = Gate<BN, kPair>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * kMaxStages + 4];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  volatile int* abort = &abort_flag;
  const uint32_t S = p.stages, x_bytes = static_cast<uint32_t>(p.box_rows) * kCols * 2, box_bytes = x_bytes + G::kWBytes;
  const uint32_t stage_bytes = G::kSub * box_bytes;
  const uint32_t tiles = smem_u32(smem), full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages;
  const uint32_t tfull0 = empty0 + 8 * kMaxStages, tempty0 = tfull0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  constexpr int kCtas = kPair ? 2 : 1;
  const int rank = blockIdx.x % (p.splits * kCtas), unit = blockIdx.x / (p.splits * kCtas);
  const int side = kPair ? rank & 1 : 0, split = rank / kCtas;
  const int e0 = unit % p.n_tiles * BN;
  const int64_t t0 = (static_cast<int64_t>(unit / p.n_tiles) * kCtas + side) * kTile;
  // this rank's blocks of 128 columns
  const int blocks = (p.H + 127) / 128;
  const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * split / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(blocks) * (split + 1) / p.splits);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, kCtas * G::kEpi);
    }
    *abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(smem_u32(&tmem_slot), G::kTmem);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&tmem_slot), G::kTmem);
      tmem_relinquish();
    }
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (kPair) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return kPair ? mbar_wait_bounded_cluster(bar, parity, abort, p.err, p.wait_limit_ns)
                 : mbar_wait_bounded(bar, parity, abort, p.err, p.wait_limit_ns);
  };
  const int rows = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kTile), p.T - t0))), cols = min(BN, p.E - e0);
  const bool wide = p.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0;
  // four logits of the tile's row r, from column c on
  auto put = [&](int r, int c, float4 v) {
    float* out = p.logits + (t0 + r) * p.ld + e0 + c;
    if (wide && c + 4 <= cols) {
      *reinterpret_cast<float4*>(out) = v;
    } else {
      if (c < cols) out[0] = v.x;
      if (c + 1 < cols) out[1] = v.y;
      if (c + 2 < cols) out[2] = v.z;
      if (c + 3 < cols) out[3] = v.w;
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t n = 2 / G::kSub * (kb1 - kb0), full_even = kPair ? cluster_map_shared(full0, rank - side) : full0;
      // tokens that only this tile reads leave the L2 first, the gate stays
      const uint64_t px = p.n_tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_normal(), pw = l2_policy_evict_last();
      uint32_t it = 0, s = 0, ph = 1;
      for (; it < n; ++it) {
        if (!wait(empty0 + 8 * s, ph)) break;
        if (side == 0) mbar_arrive_expect_tx(full0 + 8 * s, kCtas * stage_bytes);
#pragma unroll
        for (int i = 0; i < G::kSub; ++i) {
          const int32_t col = (2 * kb0 + static_cast<int32_t>(it) * G::kSub + i) * kCols;
          const uint32_t to = tiles + s * stage_bytes + i * box_bytes;
          if constexpr (kPair) {
            tma_load_2d_pair(to, &tmX, full_even + 8 * s, col, static_cast<int32_t>(t0), px);
            tma_load_2d_pair(to + x_bytes, &tmW, full_even + 8 * s, col, e0 + side * G::kWRows, pw);
          } else {
            tma_load_2d(to, &tmX, full0 + 8 * s, col, static_cast<int32_t>(t0));
            tma_load_2d(to + x_bytes, &tmW, full0 + 8 * s, col, e0);
          }
        }
        if (++s == S) {
          s = 0;
          ph ^= 1;
        }
      }
      if (it < n)     // let the copies already issued land before the CTA exits
        for (uint32_t j = it > S ? it - S : 0; j < it; ++j) {
          int dummy = 0;
          mbar_wait_bounded(full0 + 8 * (j % S), (j / S) & 1, &dummy, nullptr, p.wait_limit_ns / 10);
        }
    }
  } else if (warp == 1) {
    if (lane == 0 && side == 0) {
      constexpr uint32_t idesc = gate_idesc(F16, kTile * kCtas, BN);
      const uint16_t both = static_cast<uint16_t>(3u << rank);
      uint32_t s = 0, ph = 0, done = 0;
      bool ok = true;
      for (int kb = kb0; ok && kb < kb1; kb += kRun, ++done) {
        const uint32_t b = done & 1;
        ok = wait(tempty0 + 8 * b, ((done >> 1) & 1) ^ 1);
        const int n = 2 / G::kSub * min(kRun, kb1 - kb);
        for (int i = 0; ok && i < n; ++i) {
          ok = wait(full0 + 8 * s, ph);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < G::kSub; ++j) {
            const uint32_t at = tiles + s * stage_bytes + j * box_bytes;
            const uint64_t ad = sdesc_kmajor_sw128(at), bd = sdesc_kmajor_sw128(at + x_bytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)      // 16 columns, 32 bytes, an MMA: +2 in the 16-byte address field
              umma_f16<kPair>(tmem + b * BN, ad + 2 * k, bd + 2 * k, idesc, i | j | k ? 1u : 0u);
          }
          if constexpr (kPair) umma_commit_pair(empty0 + 8 * s, both); else umma_commit(empty0 + 8 * s);
          if (++s == S) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok) {
          if constexpr (kPair) umma_commit_pair(tfull0 + 8 * b, both); else umma_commit(tfull0 + 8 * b);
        }
      }
      if (!ok) {   // wait for the MMAs in flight before TMEM is freed
        int dummy = 0;
        const uint32_t j = s == 0 ? S - 1 : s - 1;
        mbar_wait_bounded(empty0 + 8 * j, s == 0 ? ph ^ 1 : ph, &dummy, nullptr, p.wait_limit_ns / 10);
      }
    }
    __syncwarp();
    if constexpr (!kPair) {
      // Given back before the cluster is waited for: a small CTA finds room beside a GEMM's, which may
      // want all of the SM's tensor memory while the cluster's other CTAs want some of another SM's.
      named_sync(kTmemBarrier, 32 + 32 * G::kEpi);
      tc_fence_after();
      tmem_dealloc(tmem, G::kTmem);
    }
  } else {
    const int q = warp & 3, g = (warp - 2) >> 2;
    float2 acc[G::kPer / 2];
#pragma unroll
    for (int i = 0; i < G::kPer / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
    const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16) + g * 64;
    const uint32_t tempty = kPair ? cluster_map_shared(tempty0, rank - side) : tempty0;
    bool ok = true;
    uint32_t done = 0;
    for (int kb = kb0; kb < kb1; kb += kRun, ++done) {
      const uint32_t b = done & 1;
      int got = 1;
      if (lane == 0) got = wait(tfull0 + 8 * b, (done >> 1) & 1);
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < G::kPer; c += G::kLoad) {
        constexpr int n = G::kLoad;
        uint32_t r[n];
        if constexpr (n == 32) tmem_ld_32x32b_x32(from + b * BN + c, r); else tmem_ld_32x32b_x16(from + b * BN + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
          float2& a = acc[c / 2 + i];
          a = __fadd2_rn(a, make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_cluster(tempty + 8 * b); else mbar_arrive(tempty + 8 * b);
      }
    }
    if constexpr (!kPair) {
      tc_fence_before();
      named_arrive(kTmemBarrier, 32 + 32 * G::kEpi);
    }
    // The part goes to shared memory, over the ring: with the last accumulator full every
    // copy has landed and every MMA has read its stage.
    if (ok) {
      float* part = reinterpret_cast<float*>(smem);
      if (q * 32 + lane < p.box_rows) {
        float* row = part + (q * 32 + lane) * G::kLd + g * 64;
#pragma unroll
        for (int i = 0; i < G::kPer / 4; ++i)
          *reinterpret_cast<float4*>(row + 4 * i) = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
      }
      __syncwarp();
      if (p.splits == 1) {     // each warp stores what it has, whole rows of it at a time
        constexpr int n = G::kPer / 4;
#pragma unroll 4
        for (int i = lane; i < 32 * n; i += 32) {
          const int r = q * 32 + i / n, c = g * 64 + i % n * 4;
          if (r < rows) put(r, c, *reinterpret_cast<const float4*>(part + r * G::kLd + c));
        }
      }
    }
  }
  __syncwarp();
  if (p.splits > 1) {
    cluster_sync_all();
    // each split adds its share of the tile, the parts in the order of the splits
    const int items = rows * (BN / 4);
    const int i0 = static_cast<int>(static_cast<int64_t>(items) * split / p.splits);
    const int i1 = static_cast<int>(static_cast<int64_t>(items) * (split + 1) / p.splits);
    for (int i = i0 + threadIdx.x; i < i1; i += G::kThreadCount) {
      const int r = i / (BN / 4), c = i % (BN / 4) * 4;
      const uint32_t at = tiles + (r * G::kLd + c) * 4;
      float4 part[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < p.splits) part[k] = ld_cluster_f32x4(cluster_map_shared(at, k * kCtas + side));
      float4 v = part[0];
#pragma unroll
      for (int k = 1; k < 8; ++k)
        if (k < p.splits) {
          v.x += part[k].x;
          v.y += part[k].y;
          v.z += part[k].z;
          v.w += part[k].w;
        }
      put(r, c, v);
    }
    __syncwarp();
  }
  tc_fence_before();
  // Parts are read, and barriers arrived at, by other CTAs: none leaves before the others are
  // done with it.  What they read has been stored by now, so no order of memory is asked for,
  // which would have each CTA wait for its stores.
  if (kPair || p.splits > 1) cluster_sync_relaxed();
  if constexpr (kPair) {
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc_pair(tmem, G::kTmem);
    }
  }
}

// Up to 16 tokens: a tile would be idle, and what counts is how soon the gate's rows are
// here.  A CTA takes EB experts whole, its threads 8 columns at a time.
constexpr int kFewThreads = 256;
constexpr int kFewTokens = 16;

template <int TT, int EB, bool F16>
__global__ void __launch_bounds__(kFewThreads) gate_few_kernel(const __grid_constant__ moe_gate_desc d) {
  __shared__ float sums[kFewThreads / 32][TT * EB];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = blockIdx.x * EB;
  grid_dependency_wait();
  grid_launch_dependents();
  float2 acc[TT][EB];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int e = 0; e < EB; ++e) acc[t][e] = make_float2(0.0f, 0.0f);
  const uint16_t* x = static_cast<const uint16_t*>(d.x);
  const uint16_t* w = static_cast<const uint16_t*>(d.w);
  const int T = static_cast<int>(d.T);
#pragma unroll TT * EB <= 4 ? 4 : 2
  for (int h = 8 * threadIdx.x; h < d.H; h += 8 * kFewThreads) {
    uint4 wv[EB], xv[TT];
#pragma unroll
    for (int e = 0; e < EB; ++e) wv[e] = __ldg(reinterpret_cast<const uint4*>(w + min(e0 + e, d.E - 1) * d.w_ld + h));
#pragma unroll
    for (int t = 0; t < TT; ++t) xv[t] = __ldg(reinterpret_cast<const uint4*>(x + min(t, T - 1) * d.x_ld + h));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      auto word = [&](const uint4& v) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
      float2 wf[EB];
#pragma unroll
      for (int e = 0; e < EB; ++e) wf[e] = pair_to_float<F16>(word(wv[e]));
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const float2 xf = pair_to_float<F16>(word(xv[t]));
#pragma unroll
        for (int e = 0; e < EB; ++e) acc[t][e] = __ffma2_rn(xf, wf[e], acc[t][e]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int e = 0; e < EB; ++e) {
      float v = acc[t][e].x + acc[t][e].y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) sums[warp][t * EB + e] = v;
    }
  __syncthreads();
  if (threadIdx.x < TT * EB) {
    float v = sums[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kFewThreads / 32; ++i) v += sums[i][threadIdx.x];
    const int t = threadIdx.x / EB, e = e0 + threadIdx.x % EB;
    if (t < T && e < d.E) d.logits[t * d.logits_ld + e] = v;
  }
}

template <int TT, bool F16>
int launch_few(const moe_gate_desc& d, cudaStream_t st) {
  // a CTA for every SM, and no more than two of them while the sums fit a thread's registers
  const int sms = num_sms();
  if (d.E <= sms) return launch_pdl(gate_few_kernel<TT, 1, F16>, dim3(d.E), dim3(kFewThreads), 0, st, d);
  if (d.E <= 2 * sms || TT > 8) return launch_pdl(gate_few_kernel<TT, 2, F16>, dim3((d.E + 1) / 2), dim3(kFewThreads), 0, st, d);
  if constexpr (TT <= 8) return launch_pdl(gate_few_kernel<TT, 4, F16>, dim3((d.E + 3) / 4), dim3(kFewThreads), 0, st, d);
  return MOE_ERR_UNSUPPORTED;
}

// A choice of tile and split, and what it takes.
struct GatePlan {
  int bn, splits, stages;
  bool pair;
  size_t smem;
  int64_t ctas;
};

size_t gate_smem(int bn, bool pair, int box_rows, int stages) {
  // the MMA reads 128 rows of tokens whether the copy brought them or not: behind the last
  // stage there is room for them; and the parts fit over the ring
  const size_t box = static_cast<size_t>(box_rows + (pair ? bn / 2 : bn)) * kCols * 2;
  const size_t ring = stages * (bn <= 128 ? 2 : 1) * box + (box < kXBytes ? kXBytes - box : 0);
  return 1024 + std::max(ring, static_cast<size_t>(box_rows) * (bn + 4) * 4);
}

// Estimated clock cycles of the choices, the least of them: a CTA takes in some 45 bytes a
// cycle, 1500 cycles after it asked, multiplies 128 x bn x 64 in 2 bn, and costs a few
// thousand to start and end.  Two CTAs share an SM where their shared memory lets them: so it
// counts for every tile, although from BN = 128 on their registers (146 x 320, 96 x 576) never do.  Swept against every choice (17 to 6000 tokens; 8, 64, 160, 256
// and 512 experts, 70 sizes): the one taken is within 5% of the fastest at 59 of them, 26%
// slower at worst (700 tokens by 512 experts, 11.5 us for 9.1).
GatePlan plan_gate(int64_t T, int E, int H, int box_rows, int sms) {
  GatePlan best{};
  double least = 1e300;
  const int blocks = (H + 127) / 128;
  for (int pair = 0; pair < 2; ++pair)
    for (int bn = 16; bn <= 256; bn *= 2)
      for (int splits = 1; splits <= 8 && (splits == 1 || splits <= blocks); splits *= 2) {
        const int cluster = splits << pair;
        if (cluster > 8 || (pair && (bn != 256 || T <= kTile)) || (bn > 16 && bn / 2 >= E)) continue;
        const int64_t n_tiles = (E + bn - 1) / bn, m_tiles = (T + (kTile << pair) - 1) / (kTile << pair);
        const int64_t ctas = m_tiles * n_tiles * cluster;
        const int sub = bn <= 128 ? 2 : 1;
        const double stage = sub * (box_rows + (pair ? bn / 2 : bn)) * 128.0;
        const int n = 2 / sub * ((blocks + splits - 1) / splits);
        for (const double room_for : {98304.0, 196608.0}) {       // rings of which two fit an SM, or one
          const int stages = std::max(1, std::min({kMaxStages, static_cast<int>(room_for / stage), n}));
          const size_t smem = gate_smem(bn, pair, box_rows, stages);
          if (smem > kMaxSmemPerBlock) continue;
          const int on_sm = smem <= 110 * 1024 ? 2 : 1;
          // clusters that an even share of a GPC's SMs does not hold leave SMs idle
          const int64_t room = cluster <= 2 ? sms : cluster == 4 ? sms - sms / 19 : sms - sms / 19 * 4;
          const int64_t waves = (ctas + room * on_sm - 1) / (room * on_sm);
          const double shared = ctas > room && on_sm == 2 ? 2.0 : 1.0, feed = shared * stage / 45.0;
          const double step = std::max({feed, shared * 2.0 * bn * sub, 300.0 * sub, (1500.0 + feed) / stages});
          const double rows = std::min<int64_t>(kTile, T);
          const double end = 3000.0 + (cluster > 1 ? 1000.0 : 0.0) + rows * bn * 4.0 / (splits > 1 ? 32.0 : 40.0);
          const double cycles = waves * (end + n * step);
          if (cycles < least) {
            least = cycles;
            best = GatePlan{bn, splits, stages, pair != 0, smem, ctas};
          }
        }
      }
  return best;
}

template <int BN, bool kPair, bool F16>
int launch_gate(const GatePlan& plan, const CUtensorMap& x, const CUtensorMap& w, const GateArgs& p, cudaStream_t st) {
  using G = Gate<BN, kPair>;
  if (int rc = prepare_kernel(gate_kernel<BN, kPair, F16>, plan.smem, false)) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.ctas));
  cfg.blockDim = dim3(G::kThreadCount);
  cfg.dynamicSmemBytes = plan.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = plan.splits * (kPair ? 2 : 1);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gate_kernel<BN, kPair, F16>, x, w, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <bool F16>
int run_gate(const moe_gate_desc& d, cudaStream_t st) {
  if (d.T == 1) return launch_few<1, F16>(d, st);
  if (d.T == 2) return launch_few<2, F16>(d, st);
  if (d.T <= 4) return launch_few<4, F16>(d, st);
  if (d.T <= 8) return launch_few<8, F16>(d, st);
  if (d.T <= kFewTokens) return launch_few<16, F16>(d, st);
  const int box_rows = static_cast<int>(std::min<int64_t>(kTile, (d.T + 7) / 8 * 8));
  const GatePlan plan = plan_gate(d.T, d.E, d.H, box_rows, num_sms());
  if (plan.ctas > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const GateArgs p{d.logits, d.logits_ld, d.T, d.err, d.E, d.H, plan.splits, (d.E + plan.bn - 1) / plan.bn, box_rows, plan.stages, kWaitLimitNs};
  CUtensorMap x, w;
  if (int rc = make_tmap_b16_sw128(&x, d.x, d.T, d.H, 2 * d.x_ld, box_rows)) return rc;
  if (int rc = make_tmap_b16_sw128(&w, d.w, d.E, d.H, 2 * d.w_ld, plan.pair ? plan.bn / 2 : plan.bn)) return rc;
  if (plan.pair) return launch_gate<256, true, F16>(plan, x, w, p, st);
  switch (plan.bn) {
    case 256: return launch_gate<256, false, F16>(plan, x, w, p, st);
    case 128: return launch_gate<128, false, F16>(plan, x, w, p, st);
    case 64: return launch_gate<64, false, F16>(plan, x, w, p, st);
    case 32: return launch_gate<32, false, F16>(plan, x, w, p, st);
    default: return launch_gate<16, false, F16>(plan, x, w, p, st);
  }
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
  const int64_t out = 4 * ((d->T - 1) * d->logits_ld + d->E);
  MOE_CHECK_ARG(!memory_overlaps(d->logits, out, d->x, 2 * ((d->T - 1) * d->x_ld + d->H)) &&
                !memory_overlaps(d->logits, out, d->w, 2 * ((d->E - 1ll) * d->w_ld + d->H)));
  if (int rc = check_device()) return rc;
  return d->dtype == MOE_DTYPE_F16 ? run_gate<true>(*d, as_stream(stream)) : run_gate<false>(*d, as_stream(stream));
}
