// The router's logits: tokens times the gate's rows, fp32 sums (moe_gate).
//
//   logits[t, e] = sum_h x[t, h] * w[e, h]
//
// A skinny product: with few tokens it reads the gate (3.7 MB for 256 experts of
// hidden 7168) and should take as long as launching it; with many it reads the
// tokens, 256 multiply-adds a value, which is where GB300's tensor cores and its
// memory take equally long.  So one kernel on the tensor cores (tcgen05, 128 tokens
// by BN experts a CTA) whose tile and split follow the number of tokens:
//
//  * many tokens: BN = 256, so that a token's row is read once for 256 experts;
//  * few: the hidden dimension is split over a cluster of up to 8 CTAs, and then the
//    experts over narrower tiles, until there is a CTA for every SM.  The cluster
//    adds its parts through distributed shared memory, in the order of the ranks.
//
// Warp roles: one TMA producer (ring of stages of 64 columns, 128-byte swizzle), one
// MMA issuer, and epilogue warps, four for every 64 experts.  Precision: the tensor
// cores cut what they add to a running sum, some 2^-24 of it a step, always towards
// zero; over 448 steps (hidden 7168) that is more than the logits of a router may be
// off.  So a sum runs over 128 columns only (8 steps), into one of two accumulators,
// and the epilogue warps add it in fp32, rounded to nearest, to sums in registers
// while the next 128 run.
#include <algorithm>

#include "gemm_common.cuh"


namespace moe {
namespace {

constexpr int kTile = 128;                     // tokens
constexpr int kCols = 64;                      // columns of a stage: 128 bytes, the swizzle's row
constexpr uint32_t kXBytes = kTile * kCols * 2;

constexpr int kMaxStages = 16;

// BN experts a tile; kPair: two CTAs share the tile's gate rows and 256 tokens.
template <int BN, bool kPair>
struct Gate {
  static constexpr int kWRows = kPair ? BN / 2 : BN;         // gate rows that a CTA loads
  static constexpr uint32_t kWBytes = kWRows * kCols * 2;
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

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// A CTA's place: `rank` in its cluster of splits (x 2 in pairs) CTAs; in a pair the even
// CTA issues the MMAs of both (M = 256: its own 128 tokens and the odd one's), with half of
// the gate's rows in each one's shared memory.  The odd CTA's warp 1 tells the even one of
// its full stages; commits arrive in both, the epilogue warps of both at the even one.
template <int BN, bool kPair, bool F16>
__global__ void __launch_bounds__(Gate<BN, kPair>::kThreadCount, 1)
    gate_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const GateArgs p) {
  using G = Gate<BN, kPair>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[3 * kMaxStages + 4];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  volatile int* abort = &abort_flag;
  const uint32_t S = p.stages, x_bytes = static_cast<uint32_t>(p.box_rows) * kCols * 2, stage_bytes = x_bytes + G::kWBytes;
  const uint32_t tiles = smem_u32(smem), full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages, pfull0 = empty0 + 8 * kMaxStages;
  const uint32_t tfull0 = pfull0 + 8 * kMaxStages, tempty0 = tfull0 + 16;
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
      mbar_init(pfull0 + 8 * s, 1);
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

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t n = 2 * (kb1 - kb0);
      uint32_t it = 0, s = 0, ph = 1;
      for (; it < n; ++it) {
        if (!mbar_wait_bounded(empty0 + 8 * s, ph, abort, p.err, p.wait_limit_ns)) break;
        mbar_arrive_expect_tx(full0 + 8 * s, stage_bytes);
        const int32_t col = (2 * kb0 + static_cast<int32_t>(it)) * kCols;
        tma_load_2d(tiles + s * stage_bytes, &tmX, full0 + 8 * s, col, static_cast<int32_t>(t0));
        tma_load_2d(tiles + s * stage_bytes + x_bytes, &tmW, full0 + 8 * s, col, e0 + side * G::kWRows);
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
      for (int kb = kb0; ok && kb < kb1; ++kb, ++done) {
        const uint32_t b = done & 1;
        ok = kPair ? mbar_wait_bounded_cluster(tempty0 + 8 * b, ((done >> 1) & 1) ^ 1, abort, p.err, p.wait_limit_ns)
                   : mbar_wait_bounded(tempty0 + 8 * b, ((done >> 1) & 1) ^ 1, abort, p.err, p.wait_limit_ns);
        for (int half = 0; ok && half < 2; ++half) {
          ok = mbar_wait_bounded(full0 + 8 * s, ph, abort, p.err, p.wait_limit_ns) &&
               (!kPair || mbar_wait_bounded_cluster(pfull0 + 8 * s, ph, abort, p.err, p.wait_limit_ns));
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = sdesc_kmajor_sw128(tiles + s * stage_bytes), bd = sdesc_kmajor_sw128(tiles + s * stage_bytes + x_bytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)      // 16 columns, 32 bytes, an MMA: +2 in the 16-byte address field
            umma_f16<kPair>(tmem + b * BN, ad + 2 * k, bd + 2 * k, idesc, half | k ? 1u : 0u);
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
    } else if (kPair && lane == 0) {
      const uint32_t to = cluster_map_shared(pfull0, rank - 1);
      uint32_t s = 0, ph = 0;
      for (int it = 2 * kb0; it < 2 * kb1; ++it) {
        if (!mbar_wait_bounded(full0 + 8 * s, ph, abort, p.err, p.wait_limit_ns)) break;
        mbar_arrive_cluster(to + 8 * s);
        if (++s == S) {
          s = 0;
          ph ^= 1;
        }
      }
    }
  } else {
    const int q = warp & 3, g = (warp - 2) >> 2;
    float2 acc[G::kPer / 2];
#pragma unroll
    for (int i = 0; i < G::kPer / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
    const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16) + g * 64;
    const uint32_t tempty = kPair ? cluster_map_shared(tempty0, rank - side) : tempty0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      const uint32_t done = kb - kb0, b = done & 1;
      int got = 1;
      if (lane == 0) got = mbar_wait_bounded(tfull0 + 8 * b, (done >> 1) & 1, abort, p.err, p.wait_limit_ns);
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
    // The part goes to shared memory, over the ring: with the last accumulator full every
    // copy has landed and every MMA has read its stage.
    if (ok && q * 32 + lane < p.box_rows) {
      float* row = reinterpret_cast<float*>(smem) + (q * 32 + lane) * G::kLd + g * 64;
#pragma unroll
      for (int i = 0; i < G::kPer / 4; ++i)
        *reinterpret_cast<float4*>(row + 4 * i) = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync_all(); else __syncthreads();
  // each split adds its share of the tile, the parts in the order of the splits
  const int rows = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kTile), p.T - t0))), cols = min(BN, p.E - e0);
  const int items = rows * (BN / 4);
  const int i0 = static_cast<int>(static_cast<int64_t>(items) * split / p.splits);
  const int i1 = static_cast<int>(static_cast<int64_t>(items) * (split + 1) / p.splits);
  const bool wide = p.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0;
  for (int i = i0 + threadIdx.x; i < i1; i += G::kThreadCount) {
    const int r = i / (BN / 4), c = i % (BN / 4) * 4;
    if (c >= cols) continue;
    const uint32_t at = tiles + (r * G::kLd + c) * 4;
    float4 v;
    if (p.splits == 1) {
      v = *reinterpret_cast<const float4*>(smem + (r * G::kLd + c) * 4);
    } else {
      float4 part[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < p.splits) part[k] = ld_cluster_f32x4(cluster_map_shared(at, k * kCtas + side));
      v = part[0];
#pragma unroll
      for (int k = 1; k < 8; ++k)
        if (k < p.splits) {
          v.x += part[k].x;
          v.y += part[k].y;
          v.z += part[k].z;
          v.w += part[k].w;
        }
    }
    float* out = p.logits + (t0 + r) * p.ld + e0 + c;
    if (wide && c + 4 <= cols) {
      *reinterpret_cast<float4*>(out) = v;
    } else {
      out[0] = v.x;
      if (c + 1 < cols) out[1] = v.y;
      if (c + 2 < cols) out[2] = v.z;
      if (c + 3 < cols) out[3] = v.w;
    }
  }
  tc_fence_before();
  if (kPair || p.splits > 1) cluster_sync_all(); else __syncthreads();   // parts are read, and barriers arrived at, by others
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair) tmem_dealloc_pair(tmem, G::kTmem); else tmem_dealloc(tmem, G::kTmem);
  }
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
  const size_t stage = static_cast<size_t>(box_rows + (pair ? bn / 2 : bn)) * kCols * 2;
  const size_t ring = stages * stage + (stage < kXBytes ? kXBytes - stage : 0);
  return 1024 + std::max(ring, static_cast<size_t>(box_rows) * (bn + 4) * 4);
}

// Estimated clock cycles of the choices, the least of them: a CTA takes in some 56 bytes a
// cycle and multiplies 128 x bn x 64 in 2 bn, and costs a few thousand to start and end.
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
        const double stage = (box_rows + (pair ? bn / 2 : bn)) * 128.0;
        const int n = 2 * ((blocks + splits - 1) / splits);
        int stages = std::min(kMaxStages, static_cast<int>((bn >= 128 ? 196608.0 : 98304.0) / stage));
        stages = std::max(2, std::min(stages, n));
        const size_t smem = gate_smem(bn, pair, box_rows, stages);
        const int on_sm = smem <= 110 * 1024 ? 2 : 1;
        // clusters that an even share of a GPC's SMs does not hold leave SMs idle
        const int64_t room = cluster <= 2 ? sms : cluster == 4 ? sms - sms / 19 : sms - sms / 19 * 4;
        const int64_t waves = (ctas + room * on_sm - 1) / (room * on_sm);
        const double shared = ctas > room && on_sm == 2 ? 2.0 : 1.0;
        const double step = std::max({shared * stage / 56.0, shared * 2.0 * bn, 200.0});
        const double rows = std::min<int64_t>(kTile, T);
        const double end = 3000.0 + (cluster > 1 ? 1000.0 : 0.0) + rows * bn * 4.0 / (splits > 1 ? 20.0 : 40.0);
        const double cycles = waves * (end + n * step);
        if (cycles < least) {
          least = cycles;
          best = GatePlan{bn, splits, stages, pair != 0, smem, ctas};
        }
      }
  return best;
}

template <int BN, bool kPair, bool F16>
int launch_gate(const moe_gate_desc& d, const GatePlan& plan, const CUtensorMap& x, const CUtensorMap& w, const GateArgs& p, cudaStream_t st) {
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
  const int box_rows = static_cast<int>(std::min<int64_t>(kTile, (d.T + 7) / 8 * 8));
  const GatePlan plan = plan_gate(d.T, d.E, d.H, box_rows, num_sms());
  if (plan.ctas > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const GateArgs p{d.logits, d.logits_ld, d.T, d.err, d.E, d.H, plan.splits, (d.E + plan.bn - 1) / plan.bn, box_rows, plan.stages, kWaitLimitNs};
  CUtensorMap x, w;
  if (int rc = make_tmap_b16_sw128(&x, d.x, d.T, d.H, 2 * d.x_ld, box_rows)) return rc;
  if (int rc = make_tmap_b16_sw128(&w, d.w, d.E, d.H, 2 * d.w_ld, plan.pair ? plan.bn / 2 : plan.bn)) return rc;
  if (plan.pair) return launch_gate<256, true, F16>(d, plan, x, w, p, st);
  switch (plan.bn) {
    case 256: return launch_gate<256, false, F16>(d, plan, x, w, p, st);
    case 128: return launch_gate<128, false, F16>(d, plan, x, w, p, st);
    case 64: return launch_gate<64, false, F16>(d, plan, x, w, p, st);
    case 32: return launch_gate<32, false, F16>(d, plan, x, w, p, st);
    default: return launch_gate<16, false, F16>(d, plan, x, w, p, st);
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
  if (int rc = check_device()) return rc;
  return d->dtype == MOE_DTYPE_F16 ? run_gate<true>(*d, as_stream(stream)) : run_gate<false>(*d, as_stream(stream));
}
