// mx_gemm_few.cu - the product with its gate, act(A . G^T) (A . U^T), where its tiles
// do not fill the GPU: one token to a few hundred.
//
// The weights are then what is read (2 F K bytes), or the tiles are too few to keep
// the SMs busy. The product is therefore taken the other way round: 128 rows of the gate
// and the same 128 of the up projection are the MMA's M (two accumulators), up to kN
// tokens its N, so no tensor-core rows go to tokens that do not exist; and the
// contraction is cut over the CTAs of a cluster, so that there are as many CTAs as it takes
// to have enough loads in flight. Each CTA runs its K blocks through a ring of
// shared-memory stages (TMA, one barrier each way; the scale atoms go to tensor memory
// from the MMA's own thread, in order before the MMAs that use them), leaves its FP32
// sums in its shared memory, and the cluster's CTAs take a share of the tokens each
// and add the partial sums in the order of the contraction: the same bits every time.
//
// Every wait is bounded in wall time; on expiry the CTA records MX_ERR_TIMEOUT, waits
// for its own copies and MMAs, and its tile comes out as NaN. A CTA holds tensor memory
// while it waits for the cluster's others; every kernel here that takes all of an SM's
// tensor memory takes nearly all of its shared memory too, so none can hold it on a
// shared SM and wait for one of these in turn; and no set of these that shares an SM asks
// for more than it has.
//
// Measured, weights from HBM: one token, F 10944, K 2048: 11.3 us (4.0 TB/s; the least
// launch of this kernel takes 3.5), F 18432, K 7168: 44 us (6.0 TB/s).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "mx_act.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kRows = 128;    // weight rows of a tile: the MMA's M
constexpr int kBK = 128;      // K bytes of a stage
constexpr int kThreads = 256;
constexpr int kMaxSplit = 8;  // CTAs of a cluster

template <int kN>
struct FewCfg {
  static constexpr int kStages = kN == 128 ? 4 : 2;
  static constexpr int kCtas = kN == 128 ? 1 : kN == 16 ? 3 : 2;  // of an SM
  static constexpr uint32_t kWeight = kRows * kBK;
  static constexpr uint32_t kTokens = kN * kBK;
  static constexpr uint32_t kStage = 2 * kWeight + kTokens;
  static constexpr uint32_t kScales = 3 * 512;
  static constexpr uint32_t kTx = kStage + kScales;
  static constexpr uint32_t kSfCol0 = 2 * kN;  // behind the two accumulators
  static constexpr uint32_t kTmemCols = kN == 16 ? 64 : kN == 32 ? 128 : kN == 64 ? 256 : 512;
  static_assert(kSfCol0 + kStages * 12 <= kTmemCols, "tensor memory");
  static_assert(2 * kN * kRows * 4 <= kStages * kStage, "the partial sums take the ring's place");
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kTx;
  static_assert(kCtas * (kSmem + 2048) <= 233472, "shared memory");
  static_assert(kCtas * kTmemCols <= 512, "tensor memory");
};

struct FewArgs {
  CUtensorMap gate, up, tokens;
  const uint8_t *gate_scale, *up_scale, *token_scale;
  int64_t M, F;
  __nv_bfloat16* c;
  int64_t ldc;
  __nv_bfloat16* preact;  // [M, 2F], gate first; null: not kept
  int64_t ld_preact;
  int32_t ka;             // K blocks of 128
  int32_t tiles_f;
  int32_t split;          // CTAs of a cluster
  int32_t act;
  int32_t vec;            // 1: pieces of four columns are 8-byte aligned in both outputs
  int* dev_status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void give_up(const FewArgs& p, volatile int32_t* abort_flag) {
  if (*abort_flag == 0) {
    *abort_flag = 1;
    if (p.dev_status) atomicExch(p.dev_status, static_cast<int>(MX_ERR_TIMEOUT));
  }
}

__device__ __forceinline__ bool wait_or_give_up(uint64_t* bar, uint32_t parity, const FewArgs& p, volatile int32_t* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > p.timeout_ns) {
      give_up(p, abort_flag);
      return false;
    }
  }
}

__device__ __forceinline__ float2 activate(int act, float2 z) {
  if (act == MX_ACT_SILU) return act_value<MX_ACT_SILU>(z);
  if (act == MX_ACT_GELU) return act_value<MX_ACT_GELU>(z);
  if (act == MX_ACT_RELU) return act_value<MX_ACT_RELU>(z);
  return z;
}

// Four columns of a row in BF16; `n` of them exist.
__device__ __forceinline__ void store_four(__nv_bfloat16* dst, float2 a, float2 b, int n, bool vec) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(b.x, b.y);
  if (vec && n >= 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    return;
  }
  if (n > 0) dst[0] = lo.x;
  if (n > 1) dst[1] = lo.y;
  if (n > 2) dst[2] = hi.x;
  if (n > 3) dst[3] = hi.y;
}

template <int kN>
__global__ void __launch_bounds__(kThreads, FewCfg<kN>::kCtas) gated_few_kernel(const __grid_constant__ FewArgs p) {
  using C = FewCfg<kN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  // The same offset in every CTA of the cluster: the partial sums are read by it.
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* scales = smem + S * C::kStage;
  __shared__ uint64_t full_bar[S], empty_bar[S], acc_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int32_t s_abort_flag;
  volatile int32_t* s_abort = &s_abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t split = p.split, rank = static_cast<int32_t>(blockIdx.x) % split, tile = static_cast<int32_t>(blockIdx.x) / split;
  const int32_t tf = tile % p.tiles_f, tt = tile / p.tiles_f;
  const int32_t kb0 = static_cast<int32_t>(static_cast<int64_t>(p.ka) * rank / split);
  const int32_t kb1 = static_cast<int32_t>(static_cast<int64_t>(p.ka) * (rank + 1) / split);
  const int32_t nkb = kb1 - kb0;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&acc_bar, 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.gate);
    tma_prefetch_desc(&p.up);
    tma_prefetch_desc(&p.tokens);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_wait();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    if (lane == 0) {
      int32_t issued = 0;
      for (int32_t i = 0; i < nkb; ++i) {
        const int s = i % S;
        if (!wait_or_give_up(&empty_bar[s], ((i / S) & 1) ^ 1, p, s_abort)) break;
        const int64_t kb = kb0 + i;
        uint8_t* st = smem + s * C::kStage;
        uint8_t* sf = scales + s * C::kScales;
        mbar_arrive_expect_tx(&full_bar[s], C::kTx);
        tma_load_2d(st, &p.gate, &full_bar[s], static_cast<int32_t>(kb * kBK), tf * kRows);
        tma_load_2d(st + C::kWeight, &p.up, &full_bar[s], static_cast<int32_t>(kb * kBK), tf * kRows);
        tma_load_2d(st + 2 * C::kWeight, &p.tokens, &full_bar[s], static_cast<int32_t>(kb * kBK), tt * kN);
        bulk_load(sf, p.gate_scale + ((static_cast<int64_t>(tf) * p.ka + kb) << 9), 512, &full_bar[s]);
        bulk_load(sf + 512, p.up_scale + ((static_cast<int64_t>(tf) * p.ka + kb) << 9), 512, &full_bar[s]);
        bulk_load(sf + 1024, p.token_scale + ((static_cast<int64_t>(tt) * p.ka + kb) << 9), 512, &full_bar[s]);
        ++issued;
      }
      // The copies in flight land before the ring's memory is used again, whatever
      // the MMA's thread has waited for.
      for (int32_t i = max(0, issued - S); i < issued; ++i) mbar_wait(&full_bar[i % S], (i / S) & 1, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_mxf8_e4m3(kRows, kN);
      for (int32_t i = 0; i < nkb; ++i) {
        const int s = i % S;
        if (!wait_or_give_up(&full_bar[s], (i / S) & 1, p, s_abort)) break;
        tc_fence_after_sync();
        const uint32_t st = smem_u32(smem + s * C::kStage), sf = smem_u32(scales + s * C::kScales);
        const uint32_t sf_t = tmem + C::kSfCol0 + static_cast<uint32_t>(12 * s);
#pragma unroll
        for (int j = 0; j < 3; ++j) tc_cp_32x128b_warpx4(sf_t + 4 * j, sdesc_scale_atom(sf + 512 * j));
        const uint64_t gdesc = sdesc_kmajor_sw128(st), udesc = sdesc_kmajor_sw128(st + C::kWeight),
                       tdesc = sdesc_kmajor_sw128(st + 2 * C::kWeight);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t id = idesc_with_sf_id(idesc, k, k), more = (i | k) != 0 ? 1u : 0u;
          tc_mma_mxf8(tmem, gdesc + 2 * k, tdesc + 2 * k, id, sf_t, sf_t + 8, more);
          tc_mma_mxf8(tmem + kN, udesc + 2 * k, tdesc + 2 * k, id, sf_t + 4, sf_t + 8, more);
        }
        tc_commit(&empty_bar[s]);
      }
      tc_commit(&acc_bar);  // also on expiry: everything issued has then completed
    }
    __syncwarp();
  }
  const bool done = mbar_wait(&acc_bar, 0, p.timeout_ns);
  if (!done) give_up(p, s_abort);
  __syncthreads();  // the ring is free: its copies have landed and its MMAs are done
  const bool ok = *s_abort == 0;
  tc_fence_after_sync();

  // The sums to shared memory, [gate, up][token][weight row]; two warps share a lane
  // quarter's tokens, 16 at a time.
  const int64_t token0 = static_cast<int64_t>(tt) * kN;
  const int tokens = static_cast<int>(min64(kN, p.M - token0));
  float* part = reinterpret_cast<float*>(smem);
  {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int t = (warp >> 2) * 16; t < 2 * kN; t += 32) {  // the gate's columns, then the up projection's
      if ((t & (kN - 1)) >= tokens) continue;
      uint32_t v[16];
      tmem_ld_32x32b_x16(taddr + t, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(t + i) * kRows + row] = ok ? __uint_as_float(v[i]) : __int_as_float(0x7FFFFFFF);
    }
  }
  tc_fence_before_sync();
  if (split > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  // A warp takes a token, a lane four columns of it; the tokens are dealt to the
  // cluster's warps in turn.
  const int64_t f = static_cast<int64_t>(tf) * kRows + 4 * lane;
  const int n = static_cast<int>(min64(4, p.F - f));
  const uint32_t mine = smem_u32(part) + 16 * lane;
#pragma unroll 1
  for (int t = warp * split + rank; t < tokens; t += split * (kThreads / 32)) {
    float2 g0 = make_float2(0.0f, 0.0f), g1 = g0, u0 = g0, u1 = g0;
#pragma unroll 4
    for (int r = 0; r < split; ++r) {
      const uint32_t at = mapa_shared(mine + 4 * t * kRows, r);
      const float4 g = ld_cluster_v4(at), u = ld_cluster_v4(at + 4 * kN * kRows);
      g0 = __fadd2_rn(g0, make_float2(g.x, g.y));
      g1 = __fadd2_rn(g1, make_float2(g.z, g.w));
      u0 = __fadd2_rn(u0, make_float2(u.x, u.y));
      u1 = __fadd2_rn(u1, make_float2(u.z, u.w));
    }
    const int64_t token = token0 + t;
    store_four(p.c + token * p.ldc + f, __fmul2_rn(activate(p.act, g0), u0), __fmul2_rn(activate(p.act, g1), u1), n, p.vec);
    if (p.preact) {
      __nv_bfloat16* z = p.preact + token * p.ld_preact + f;
      store_four(z, g0, g1, n, p.vec);
      store_four(z + p.F, u0, u1, n, p.vec);
    }
  }
  if (split > 1) cluster_sync();  // nobody leaves while its sums are read
}

// Clusters of `split` CTAs that the current device runs at once with a CTA on an SM
// (which is how the runtime counts them: 76, 46, 36, 28, 23, 15, 15 for two to eight);
// asked of it once for each device. The kernel's shared memory is allowed by then.
template <int kN>
int clusters_held(int split) {
  constexpr int kDevices = 16;
  static std::atomic<int> seen[kDevices][kMaxSplit + 1];  // 0: not asked yet, else one more
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < kDevices)
    if (const int h = seen[dev][split].load(std::memory_order_relaxed)) return h - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = FewCfg<kN>::kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(split), 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int held = 0;
  if (cudaOccupancyMaxActiveClusters(&held, gated_few_kernel<kN>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    held = 0;
  }
  if (dev < kDevices) seen[dev][split].store(held + 1, std::memory_order_relaxed);
  return held;
}

template <int kN>
mx_status launch_few(const GemmLaunch& L, int min_blocks, cudaStream_t s) {
  using C = FewCfg<kN>;
  FewArgs a = {};
  mx_status st = make_operand_map(&a.gate, L.b_data, L.N / 2, L.K, L.b_ld, kRows);
  if (st == MX_OK) st = make_operand_map(&a.up, L.up_data, L.N / 2, L.K, L.up_ld, kRows);
  const WaitTest test = take_wait_test();
  if (st == MX_OK) st = make_operand_map(&a.tokens, L.a_data, L.M, L.K, L.a_ld, test.stages() ? kN / 2 : kN);
  if (st != MX_OK) return st;
  a.gate_scale = static_cast<const uint8_t*>(L.b_scale);
  a.up_scale = static_cast<const uint8_t*>(L.up_scale);
  a.token_scale = static_cast<const uint8_t*>(L.a_scale);
  a.M = L.M;
  a.F = L.N / 2;
  a.c = static_cast<__nv_bfloat16*>(L.c);
  a.ldc = L.ldc;
  a.preact = static_cast<__nv_bfloat16*>(L.epi.preact);
  a.ld_preact = L.epi.ld_preact;
  a.ka = static_cast<int32_t>((L.K + kBK - 1) / kBK);
  a.tiles_f = static_cast<int32_t>((a.F + kRows - 1) / kRows);
  a.act = L.epi.act;
  const auto aligned = [](const void* q, int64_t ld) { return (reinterpret_cast<uintptr_t>(q) & 7u) == 0 && ld % 4 == 0; };
  a.vec = aligned(L.c, L.ldc) && (!L.epi.preact || (aligned(L.epi.preact, L.epi.ld_preact) && a.F % 4 == 0));
  a.dev_status = L.dev_status;
  a.timeout_ns = test.limit();
  const auto kern = gated_few_kernel<kN>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
  if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(gated few)");
  const int64_t tiles = a.tiles_f * ((L.M + kN - 1) / kN);
  int split = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kMaxSplit, C::kCtas * sm_count() / tiles, a.ka / min_blocks})));
  while (split > 1 && C::kCtas * clusters_held<kN>(split) < tiles) --split;
  a.split = split;
  return cuda_status(launch_kernel(kern, static_cast<unsigned>(tiles * split), kThreads, C::kSmem, s, static_cast<unsigned>(split), a),
                     "mx_gemm_gated launch");
}

}  // namespace

// Taken for up to 32 tokens, and for more where a tile of 128 x 128 can have four CTAs
// with four K blocks each and they are no more than the SMs. (All run at once up to 36
// tiles; with 37 or 38 of more than 64 tokens launch_few cuts in three: F 4736, K 2048, 100
// tokens 12.0 us.) us of this kernel and of the one for whole tiles (mx_gemm.cu), weights
// from HBM:
//   F 10944, K 2048:   1 token 11.3, 17.4   32: 13.5, 16.8   64: 15.6, 13.7
//   F 18432, K 7168:   1 token 43.9, 55.9   32: 46.4, 46.5   64: 48.2, 46.8
//   F  1408, K 2048:   1 token  5.6, 10.8   64:  8.5, 10.9  333: 10.5, 10.9
//   F  2816, K 7168:   1 token 12.1, 25.4   64: 17.7, 23.8  128: 16.3, 23.9
//   F   512, K  512:   1 token  3.5,  6.5  128:  7.2,  6.6
// With weights in L2 333 tokens take 9.7 at F 1408, K 2048.
bool gated_few_applies(const GemmLaunch& L) {
  const int64_t tiles = (L.N / 2 + kRows - 1) / kRows * ((L.M + 127) / 128);
  if (L.M <= 32) return tiles * kMaxSplit <= INT32_MAX;
  return 4 * tiles <= sm_count() && L.K > 15 * kBK;
}

// CTAs of a tile: as many as can all run at once, each with at least one K block; with
// four where the tile has more than 32 tokens, whose sums are dear to join (F 1408, K
// 2048, 64 tokens: 8.5 us with four CTAs, 10.0 with eight). F 8192, K 2048, 1 token: 12.1
// us with two, 10.5 with four, 9.7 with six, 14.3 with seven, which do not all run.
mx_status launch_gated_few(const GemmLaunch& L, cudaStream_t s) {
  if (L.M <= 16) return launch_few<16>(L, 1, s);
  if (L.M <= 32) return launch_few<32>(L, 1, s);
  if (L.M <= 64) return launch_few<64>(L, 4, s);
  return launch_few<128>(L, 4, s);
}

}  // namespace mx
