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

template <int BN>
struct Gate {
  static constexpr uint32_t kWBytes = BN * kCols * 2;
  static constexpr uint32_t kStage = kXBytes + kWBytes;
  static constexpr int kStages = kStage * 8 <= 200 * 1024 ? 8 : kStage * 6 <= 200 * 1024 ? 6 : 4;
  static constexpr int kEpi = BN > 64 ? BN / 16 : 4;         // epilogue warps
  static constexpr int kPer = BN > 64 ? 64 : BN;             // experts of a warp
  static constexpr int kThreadCount = 64 + 32 * kEpi;
  static constexpr int kLd = BN + 4;                         // of the parts in shared memory, floats
  static constexpr uint32_t kTmem = BN < 16 ? 32 : 2 * BN;
  static constexpr size_t kSmem = 1024 + kStages * kStage + 8 * (2 * kStages + 4) + 16;
  static_assert(kTile * kLd * 4 <= kStages * kStage, "parts fit the ring");
  static_assert(kSmem <= kMaxSmemPerBlock, "shared memory");
};

struct GateArgs {
  float* logits;
  int64_t ld;
  int64_t T;
  int32_t* err;
  int32_t E, H, splits, n_tiles, box_rows;
  uint64_t wait_limit_ns;
};

// kind::f16 with fp32 sums, both operands K-major, f16 or bf16.
__host__ __device__ constexpr uint32_t gate_idesc(bool f16, int N) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(kTile >> 4) << 24);
}

__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int BN, bool F16>
__global__ void __launch_bounds__(Gate<BN>::kThreadCount, 1)
    gate_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const GateArgs p) {
  using G = Gate<BN>;
  constexpr int S = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * G::kStage);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 4);
  volatile int* abort = reinterpret_cast<int*>(tmem_slot + 1);
  const uint32_t tiles = smem_u32(smem), full0 = smem_u32(bars), empty0 = full0 + 8 * S, tfull0 = empty0 + 8 * S, tempty0 = tfull0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int rank = blockIdx.x % p.splits, unit = blockIdx.x / p.splits;
  const int e0 = unit % p.n_tiles * BN;
  const int64_t t0 = static_cast<int64_t>(unit / p.n_tiles) * kTile;
  // this rank's blocks of 128 columns
  const int blocks = (p.H + 127) / 128;
  const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / p.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, G::kEpi);
    }
    *abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), G::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  float2 acc[G::kPer / 2];
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t bytes = static_cast<uint32_t>(p.box_rows) * kCols * 2 + G::kWBytes;
      const uint32_t n = 2 * (kb1 - kb0);
      uint32_t it = 0;
      for (; it < n; ++it) {
        const uint32_t s = it % S;
        if (!mbar_wait_bounded(empty0 + 8 * s, ((it / S) & 1) ^ 1, abort, p.err, p.wait_limit_ns)) break;
        mbar_arrive_expect_tx(full0 + 8 * s, bytes);
        const int32_t col = (2 * kb0 + static_cast<int32_t>(it)) * kCols;
        tma_load_2d(tiles + s * G::kStage, &tmX, full0 + 8 * s, col, static_cast<int32_t>(t0));
        tma_load_2d(tiles + s * G::kStage + kXBytes, &tmW, full0 + 8 * s, col, e0);
      }
      if (it < n)     // let the copies already issued land before the CTA exits
        for (uint32_t j = it > S ? it - S : 0; j < it; ++j) {
          int dummy = 0;
          mbar_wait_bounded(full0 + 8 * (j % S), (j / S) & 1, &dummy, nullptr, p.wait_limit_ns / 10);
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = gate_idesc(F16, BN);
      uint32_t it = 0, done = 0;
      bool ok = true;
      for (int kb = kb0; ok && kb < kb1; ++kb, ++done) {
        const uint32_t b = done & 1;
        ok = mbar_wait_bounded(tempty0 + 8 * b, ((done >> 1) & 1) ^ 1, abort, p.err, p.wait_limit_ns);
        for (int half = 0; ok && half < 2; ++half, ++it) {
          const uint32_t s = it % S;
          ok = mbar_wait_bounded(full0 + 8 * s, (it / S) & 1, abort, p.err, p.wait_limit_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = sdesc_kmajor_sw128(tiles + s * G::kStage), bd = sdesc_kmajor_sw128(tiles + s * G::kStage + kXBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)      // 16 columns, 32 bytes, an MMA: +2 in the 16-byte address field
            umma_f16(tmem + b * BN, ad + 2 * k, bd + 2 * k, idesc, half | k ? 1u : 0u);
          umma_commit(empty0 + 8 * s);
        }
        if (ok) umma_commit(tfull0 + 8 * b);
      }
      if (!ok && it > 0) {   // wait for the MMAs in flight before TMEM is freed
        int dummy = 0;
        mbar_wait_bounded(empty0 + 8 * ((it - 1) % S), ((it - 1) / S) & 1, &dummy, nullptr, p.wait_limit_ns / 10);
      }
    }
  } else {
    const int q = warp & 3, g = (warp - 2) >> 2;
#pragma unroll
    for (int i = 0; i < G::kPer / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
    const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16) + g * 64;
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
      for (int c = 0; c < G::kPer; c += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(from + b * BN + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2& a = acc[c / 2 + i];
          a = __fadd2_rn(a, make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty0 + 8 * b);
    }
    // The part goes to shared memory, over the ring: with the last accumulator full every
    // copy has landed and every MMA has read its stage.
    if (ok) {
      float* row = reinterpret_cast<float*>(smem) + (q * 32 + lane) * G::kLd + g * 64;
      if (q * 32 + lane < p.box_rows) {
#pragma unroll
        for (int i = 0; i < G::kPer / 4; ++i)
          *reinterpret_cast<float4*>(row + 4 * i) = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
      }
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync_all(); else __syncthreads();
  // each rank adds its share of the tile, the ranks' parts in their order
  const int rows = static_cast<int>(min(static_cast<int64_t>(kTile), p.T - t0)), cols = min(BN, p.E - e0);
  const int items = rows * (BN / 4);
  const int i0 = static_cast<int>(static_cast<int64_t>(items) * rank / p.splits);
  const int i1 = static_cast<int>(static_cast<int64_t>(items) * (rank + 1) / p.splits);
  const bool wide = p.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0;
  for (int i = i0 + threadIdx.x; i < i1; i += G::kThreadCount) {
    const int r = i / (BN / 4), c = i % (BN / 4) * 4;
    if (c >= cols) continue;
    const uint32_t at = tiles + (r * G::kLd + c) * 4;
    float4 v = p.splits > 1 ? ld_cluster_f32x4(cluster_map_shared(at, 0)) : *reinterpret_cast<const float4*>(smem + (r * G::kLd + c) * 4);
    for (int k = 1; k < p.splits; ++k) {
      const float4 o = ld_cluster_f32x4(cluster_map_shared(at, k));
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
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
  if (p.splits > 1) cluster_sync_all(); else __syncthreads();   // parts are read by others
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kTmem);
  }
}

template <int BN, bool F16>
int launch_gate(const CUtensorMap& x, const CUtensorMap& w, const GateArgs& p, int64_t ctas, cudaStream_t st) {
  using G = Gate<BN>;
  if (int rc = prepare_kernel(gate_kernel<BN, F16>, G::kSmem, false)) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(G::kThreadCount);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gate_kernel<BN, F16>, x, w, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <bool F16>
int pick_gate(const moe_gate_desc& d, cudaStream_t st) {
  const int64_t tiles = (d.T + kTile - 1) / kTile;
  const int blocks = (d.H + 127) / 128, sms = num_sms();
  // the widest tile that the experts fill, then the split over the hidden dimension, then
  // narrower tiles, each as long as that leaves no more CTAs than SMs
  int bn = 256;
  while (bn > 16 && bn / 2 >= d.E) bn /= 2;
  auto ctas = [&](int n, int s) { return tiles * ((d.E + n - 1) / n) * s; };
  int splits = 1;
  while (splits < 8 && 2 * splits <= blocks && ctas(bn, 2 * splits) <= sms) splits *= 2;
  while (bn > 16 && ctas(bn / 2, splits) <= sms) bn /= 2;
  GateArgs p{d.logits, d.logits_ld, d.T, d.err, d.E, d.H, splits, (d.E + bn - 1) / bn,
             static_cast<int32_t>(std::min<int64_t>(kTile, (d.T + 7) / 8 * 8)), kWaitLimitNs};
  CUtensorMap x, w;
  if (int rc = make_tmap_b16_sw128(&x, d.x, d.T, d.H, 2 * d.x_ld, p.box_rows)) return rc;
  if (int rc = make_tmap_b16_sw128(&w, d.w, d.E, d.H, 2 * d.w_ld, bn)) return rc;
  const int64_t n = ctas(bn, splits);
  if (n > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  switch (bn) {
    case 256: return launch_gate<256, F16>(x, w, p, n, st);
    case 128: return launch_gate<128, F16>(x, w, p, n, st);
    case 64: return launch_gate<64, F16>(x, w, p, n, st);
    case 32: return launch_gate<32, F16>(x, w, p, n, st);
    default: return launch_gate<16, F16>(x, w, p, n, st);
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
  return d->dtype == MOE_DTYPE_F16 ? pick_gate<true>(*d, as_stream(stream)) : pick_gate<false>(*d, as_stream(stream));
}
