// mx_addnorm.cu - the residual's addition, the root-mean-square norm of the sum
// and the norm's output as MX copies, in one pass; and the backward pass.
//
//   v = x + residual,  rstd = 1 / sqrt(sum(v^2) / cols + eps),  y = v rstd weight
//   h = v rstd,  g = dy weight,  dx = dsum + rstd (g - h sum(g h) / cols),
//   dweight = sum over rows of dy h
//
// Both passes are bound by HBM: every tensor is read or written once (forward 8.06
// bytes a value with a BF16 stream and both copies, backward 10.06). What stands in
// the way is that the column copy's blocks run down 32 rows while the norm's sum
// runs along a whole row, so that 32 whole rows are needed at once: a panel of 32
// rows is split over the warps of a cluster of CTAs, 64 columns a warp (mx_block.cuh),
// and stays there in FP32 from the load to the stores. Per panel the warps exchange
// one sum for each row: warps of a CTA through shared memory, CTAs through words in
// each other's, added in a fixed order. Each warp's part of the next panel is on its
// way into shared memory (TMA, one stage per warp, its own mbarrier) as soon as the
// present one is no longer needed there.
//
// Measured, both copies (of 6787 GB/s copied): forward 16384 x 2048 50 us (79%), 8192 x
// 5120 60 us (83%), 8192 x 7168 102 us (68%), with an FP32 stream and the output in BF16
// too 163 us (75%); backward 16384 x 2048 67 us (74%, 3 of them the sum of the partial rows
// of dweight), 8192 x 7168 125 us (70%). The rest is the exchange, and clusters that leave
// SMs over: wide rows take 8 to 16 CTAs of a GPC's SMs.
//
// A wait that runs out leaves MX_ERR_TIMEOUT, and NaN in the values it was for; the
// warp loads nothing more, but takes part in every barrier.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>
#include <vector>

#include "mx_block.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kMaxCluster = 16;   // CTAs (above 8: opt-in)
constexpr int kMaxWarps = 16;     // of a CTA
constexpr int kMaxParts = 608;    // clusters of a launch (partial rows of dweight)
constexpr int kMaxSmem = 226 * 1024;

struct AddNormArgs {
  CUtensorMap a, b, c;  // forward: x, residual, -; backward: dy, sum, dsum
  const void* weight;   // null: 1
  const float* rstd_in;
  void* out;            // forward: sum (may be null); backward: dx (may be null)
  int64_t ld_out;
  __nv_bfloat16* y;     // forward: the norm's output in BF16 (may be null)
  int64_t ldy;
  float* rstd;          // forward (may be null)
  float* partial;       // backward: [cluster][cols] (may be null)
  CopyOut q;
  int64_t rows, cols;
  float eps;
  int32_t weight_f32;
  int32_t weight_vec;   // 1: the weights start on a 16-byte boundary
  int32_t has_second;   // forward: a residual; backward: dsum (2: read by the lanes themselves)
  const void* direct;   // that dsum
  int64_t ld_direct;
  int32_t warps;        // of a CTA
  int* dev_status;
  uint64_t timeout_ns;
};

// Eight bytes into a CTA's shared memory of the cluster, in one access.
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.relaxed.cluster.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}

// The rows' sums over all columns: each warp's are in lane order (lane = row). Each
// CTA sends its own to all CTAs of the cluster, a row's sum and the panel's number
// (counted from 1) in one 8-byte store, and a warp that needs a panel's sums reads
// its CTA's words until they carry that number. So nothing waits for the stores of
// outputs, as a release at cluster scope would (a barrier of the cluster per panel
// held every warp until its stores had been performed, a fifth of the time). Words
// of even and of odd panels are apart: a CTA sends a panel's sums when all its warps
// have read those of the panel before, and overwrites words two panels later, when
// it has received the sums of the panel in between from every CTA.
struct RowSums {
  uint32_t all;   // shared memory, [2 * CTAs][32] words of 8 bytes
  uint32_t part;  // [warps][32] floats, each warp's
};

// Both in dynamic shared memory, behind the stages.
__host__ __device__ constexpr uint32_t sums_bytes(uint32_t csize, uint32_t warps) { return csize * 2 * 32 * 8 + warps * 32 * 4; }

__device__ __forceinline__ RowSums sums_at(uint8_t* at, uint32_t csize) {
  const uint32_t a = smem_u32(at);
  return RowSums{a, a + csize * 2 * 32 * 8};
}

__device__ __forceinline__ void st_shared_f32(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }
__device__ __forceinline__ float ld_shared_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_shared_u64(uint32_t at) {
  uint64_t v;
  asm volatile("ld.volatile.shared.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}

// `dead`: a wait of this warp has run out. Once one of the CTA's has, the CTA sends
// nothing more (its panels come out as NaN, and the others' waits run out too):
// returns true then. kWithheld (the self test): the last CTA is sent nothing.
template <bool kWithheld>
__device__ __forceinline__ bool sums_send(const RowSums& s, float mine, bool dead, int warp, int lane, int warps, uint32_t crank,
                                          uint32_t csize, int k) {
  st_shared_f32(s.part + (warp * 32 + lane) * 4, mine);
  if (__syncthreads_or(dead)) return true;
  if (warp == 0) {
    float t = 0.0f;
    for (int w0 = 0; w0 < warps; w0 += 8) {
      float v[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) v[w] = w0 + w < warps ? ld_shared_f32(s.part + ((w0 + w) * 32 + lane) * 4) : 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += v[w];
    }
    const uint64_t word = (static_cast<uint64_t>(static_cast<uint32_t>(k) + 1u) << 32) | __float_as_uint(t);
    const uint32_t at = s.all + (((k & 1) * csize + crank) * 32 + lane) * 8;
    for (uint32_t r = 0; r < csize - (kWithheld ? 1 : 0); ++r) st_cluster_u64(mapa_shared(at, r), word);
  }
  return false;
}

// After sums_send of panel k; NaN, and dead, where the wait runs out.
__device__ __forceinline__ float sums_receive(const RowSums& s, bool& dead, int lane, uint32_t csize, int k,
                                              const AddNormArgs& p) {
  if (dead) return __int_as_float(0x7FFFFFFF);
  const uint32_t number = static_cast<uint32_t>(k) + 1u, at = s.all + ((k & 1) * csize * 32 + lane) * 8;
  const auto is_there = [&](uint64_t word) { return static_cast<uint32_t>(word >> 32) == number; };
  float t = 0.0f;
  bool there = true;
  for (uint32_t r0 = 0; r0 < csize && there; r0 += 4) {
    uint64_t word[4];
    uint64_t t0 = 0;
    do {
      there = true;
#pragma unroll
      for (uint32_t r = 0; r < 4; ++r) {
        word[r] = r0 + r < csize ? ld_shared_u64(at + (r0 + r) * 256) : static_cast<uint64_t>(number) << 32;
        there = there && is_there(word[r]);
      }
      if (!there) {
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > p.timeout_ns) break;
      }
    } while (!there);
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r) t += __uint_as_float(static_cast<uint32_t>(word[r]));
  }
  if (!there && p.dev_status) atomicExch(p.dev_status, static_cast<int>(MX_ERR_TIMEOUT));
  dead = !__all_sync(0xFFFFFFFFu, there);
  return dead ? __int_as_float(0x7FFFFFFF) : t;
}

// A lane's 8 weights (1 without any, 0 past the last column).
__device__ __forceinline__ void lane_weights(const AddNormArgs& p, int64_t c, float2 (&w)[4]) {
  const float fill = c < p.cols ? 1.0f : 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = make_float2(fill, fill);
  if (!p.weight || c >= p.cols) return;
  if (p.weight_vec) {
    if (p.weight_f32) load_row<true>(p.weight, c, w);
    else load_row<false>(p.weight, c, w);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (p.weight_f32) {
      const float* f = static_cast<const float*>(p.weight) + c + 2 * j;
      w[j] = make_float2(f[0], f[1]);
    } else {
      const __nv_bfloat16* f = static_cast<const __nv_bfloat16*>(p.weight) + c + 2 * j;
      w[j] = make_float2(__bfloat162float(f[0]), __bfloat162float(f[1]));
    }
  }
}

// One warp's load of a panel: [32 rows x 64 columns] of a tensor.
template <bool kF32>
__device__ __forceinline__ void load_box(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int c0, int row0) {
  tma_load_2d(dst, map, bar, c0, row0);
  if constexpr (kF32) tma_load_2d(dst + kF32Box, map, bar, c0 + 32, row0);
}

// Waits for a stage; false (and a status) once the limit has passed.
__device__ __forceinline__ bool stage_wait(uint64_t* bar, uint32_t parity, const AddNormArgs& p) {
  if (mbar_wait(bar, parity, p.timeout_ns)) return true;
  if (p.dev_status) atomicExch(p.dev_status, static_cast<int>(MX_ERR_TIMEOUT));
  return false;
}

__device__ __forceinline__ void fill_nan(float2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float2(__int_as_float(0x7FFFFFFF), __int_as_float(0x7FFFFFFF));
}

// kF32: the residual stream (residual and sum; backward: sum, dsum and dx) is FP32.
template <bool kF32, bool kRow, bool kCol, bool kWithheld = false>
__global__ void __launch_bounds__(32 * kMaxWarps) add_norm_kernel(const __grid_constant__ AddNormArgs p) {
  constexpr uint32_t kStage = 4096 + unit_box_bytes(kF32);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_bar[kMaxWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 7, g = lane >> 3;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();
  const int cluster = static_cast<int>(blockIdx.x / csize), clusters = static_cast<int>(gridDim.x / csize);
  const int panels = static_cast<int>((p.rows + 31) >> 5);  // rows < 2^31
  const int c0 = (static_cast<int>(crank) * p.warps + warp) * kUnitCols;
  const int c = c0 + 8 * q;
  const bool active = c0 < p.cols;
  uint8_t* stage = smem + warp * kStage;
  uint64_t* bar = &s_bar[warp];
  const RowSums sums = sums_at(smem + p.warps * kStage, csize);
  const uint32_t bytes = 4096 + (p.has_second ? (kF32 ? 8192 : 4096) : 0);

  if (lane == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  for (uint32_t i = warp; i < 2 * csize; i += p.warps)
    asm volatile("st.shared.u64 [%0], %1;" ::"r"(sums.all + (i * 32 + lane) * 8), "l"(uint64_t{0}) : "memory");
  pdl_launch_dependents();
  cluster_sync();  // every CTA of the cluster runs before one writes to it
  pdl_wait();

  auto load = [&](int panel) {
    mbar_arrive_expect_tx(bar, bytes);
    load_box<false>(stage, &p.a, bar, c0, panel * 32);
    if (p.has_second) load_box<kF32>(stage + 4096, &p.b, bar, c0, panel * 32);
  };
  if (active && lane == 0 && cluster < panels) load(cluster);
  float2 w[4];
  lane_weights(p, c, w);
  {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, n = static_cast<int64_t>(gridDim.x) * blockDim.x;
    if (kRow) zero_scale_padding(p.q.row_scale, p.rows, p.cols >> 5, p.q.row_ka, id, n);
    if (kCol) zero_scale_padding(p.q.col_scale, p.cols, p.rows >> 5, p.q.col_ka, id, n);
  }

  bool ok = true, dead = false;
  int k = 0, failed = 0;
  for (int panel = cluster; panel < panels; panel += clusters, ++k) {
    const int row0 = panel * 32;
    const int rows = static_cast<int>(min64(32, p.rows - row0));
    float2 v[8][4];
    if (active) {
      if (ok) {
        ok = __all_sync(0xFFFFFFFFu, stage_wait(bar, k & 1, p));
        failed = k;
      }
      if (ok) {
#pragma unroll
        for (int i = 0; i < 8; ++i) unit_row_bf16(stage, 8 * g + i, q, v[i]);
        if (p.has_second) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 r[4];
            unit_row<kF32>(stage + 4096, 8 * g + i, q, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = __fadd2_rn(v[i][j], r[j]);
          }
        }
        __syncwarp();
        if (lane == 0 && panel + clusters < panels) load(panel + clusters);
        __syncwarp();
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) fill_nan(v[i]);
      }
    }
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (active) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) t = __ffma2_rn(v[i][j], v[i][j], t);
        s[i] = t.x + t.y;
      }
    }
    dead = sums_send<kWithheld>(sums, fold_rows(s, lane), dead, warp, lane, p.warps, crank, csize, k);
    if (active && p.out && c < p.cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * g + i < rows) store_row<kF32>(p.out, static_cast<int64_t>(row0 + 8 * g + i) * p.ld_out + c, v[i]);
    }
    const float total = sums_receive(sums, dead, lane, csize, k, p);
    const float rstd = 1.0f / sqrtf(total / static_cast<float>(p.cols) + p.eps);
    if (crank == 0 && warp == 0 && p.rstd && lane < rows) p.rstd[row0 + lane] = rstd;
    if (!active) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = __shfl_sync(0xFFFFFFFFu, rstd, 8 * g + i);
      const float2 r2 = make_float2(r, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(__fmul2_rn(v[i][j], r2), w[j]);
    }
    if (p.y && c < p.cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * g + i < rows) store_row<false>(p.y, static_cast<int64_t>(row0 + 8 * g + i) * p.ldy + c, v[i]);
    }
    store_unit<kRow, kCol>(v, p.q, lane, row0, rows, c0, p.cols, row0);
  }
  // A warp that gave up has one load on its way at most: its stage's.
  if (active && !ok && lane == 0) mbar_wait(bar, static_cast<uint32_t>(failed & 1), p.timeout_ns);
  __syncwarp();
  cluster_sync();  // no CTA leaves while another may still write to it
}

// Up to 12 warps (kThreads 256, 384) dsum + rstd g stays in registers over the
// exchange, so that dy's and dsum's next loads are on their way during it. For more
// warps on an SM there are no registers for that (kThreads 512: 16 warps of 128): the
// values are then read once more from the stage, which is free for the next load later.
template <bool kF32, bool kRow, bool kCol, int kThreads, bool kWithheld = false>
__global__ void __launch_bounds__(kThreads, 1) add_norm_backward_kernel(const __grid_constant__ AddNormArgs p) {
  constexpr bool kHeld = kThreads < 512;
  constexpr uint32_t kStream = unit_box_bytes(kF32);
  const uint32_t streams = p.has_second == 1 ? 2 : 1, stage_bytes = 4096 + streams * kStream;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_bar[kMaxWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 7, g = lane >> 3;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();
  const int cluster = static_cast<int>(blockIdx.x / csize), clusters = static_cast<int>(gridDim.x / csize);
  const int panels = static_cast<int>((p.rows + 31) >> 5);  // rows < 2^31
  const int c0 = (static_cast<int>(crank) * p.warps + warp) * kUnitCols;
  const int c = c0 + 8 * q;
  const bool active = c0 < p.cols;
  uint8_t* stage = smem + warp * stage_bytes;
  uint64_t* bar = &s_bar[warp];
  const RowSums sums = sums_at(smem + p.warps * stage_bytes, csize);

  if (lane == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  for (uint32_t i = warp; i < 2 * csize; i += p.warps)
    asm volatile("st.shared.u64 [%0], %1;" ::"r"(sums.all + (i * 32 + lane) * 8), "l"(uint64_t{0}) : "memory");
  pdl_launch_dependents();
  cluster_sync();  // every CTA of the cluster runs before one writes to it
  pdl_wait();

  auto load = [&](int panel) {
    mbar_arrive_expect_tx(bar, 4096 + streams * (kF32 ? 8192 : 4096));
    load_box<false>(stage, &p.a, bar, c0, panel * 32);
    if (p.has_second == 1) load_box<kF32>(stage + 4096 + kStream, &p.c, bar, c0, panel * 32);
  };
  // The sum's box is read again once the rows' sums are there (in registers it would
  // cost half the warps), so its next load, of the same phase, follows later; without
  // kHeld all of a stage's do.
  auto load_sum = [&](int panel) { load_box<kF32>(stage + 4096, &p.b, bar, c0, panel * 32); };
  if (active && lane == 0 && cluster < panels) {
    load(cluster);
    load_sum(cluster);
  }
  // The next panel's statistic, a panel ahead (lane = row).
  auto load_rstd = [&](int panel) { return panel < panels && panel * 32 + lane < p.rows ? p.rstd_in[panel * 32 + lane] : 0.0f; };
  float rstd_next = load_rstd(cluster);
  float2 dweight = make_float2(0.0f, 0.0f);  // of columns 8 q + 2 g and + 1, over the panels
  {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, n = static_cast<int64_t>(gridDim.x) * blockDim.x;
    if (kRow) zero_scale_padding(p.q.row_scale, p.rows, p.cols >> 5, p.q.row_ka, id, n);
    if (kCol) zero_scale_padding(p.q.col_scale, p.cols, p.rows >> 5, p.q.col_ka, id, n);
  }

  bool ok = true, dead = false;
  int k = 0, failed = 0;
  for (int panel = cluster; panel < panels; panel += clusters, ++k) {
    const int row0 = panel * 32;
    const int rows = static_cast<int>(min64(32, p.rows - row0));
    float rstd = rstd_next;
    float2 v[8][4];  // dsum + rstd g, then dx
    const auto add_dsum = [&](int i, float2 (&to)[4]) {
      float2 d[4];
      if (p.has_second == 1) {
        unit_row<kF32>(stage + 4096 + kStream, 8 * g + i, q, d);
      } else if (8 * g + i < rows && c < p.cols) {
        load_row<kF32>(p.direct, static_cast<int64_t>(row0 + 8 * g + i) * p.ld_direct + c, d);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) to[j] = __fadd2_rn(to[j], d[j]);
    };
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (active) {
      if (ok) {
        ok = __all_sync(0xFFFFFFFFu, stage_wait(bar, k & 1, p));
        failed = k;
      }
      // Rows that are not there come as zeros; a stage that has not come makes rstd,
      // and so everything, NaN.
      if (!ok) rstd = __int_as_float(0x7FFFFFFF);
      {
        float2 w[4], dw[4];
        lane_weights(p, c, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[j] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float r = __shfl_sync(0xFFFFFFFFu, rstd, 8 * g + i);
          const float2 r2 = make_float2(r, r);
          float2 g2[4], h[4], t = make_float2(0.0f, 0.0f);
          unit_row_bf16(stage, 8 * g + i, q, g2);
          unit_row<kF32>(stage + 4096, 8 * g + i, q, h);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            g2[j] = __fmul2_rn(g2[j], r2);
            dw[j] = __ffma2_rn(g2[j], h[j], dw[j]);
            g2[j] = __fmul2_rn(g2[j], w[j]);
            t = __ffma2_rn(g2[j], h[j], t);
            if constexpr (kHeld) v[i][j] = g2[j];
          }
          s[i] = t.x + t.y;
        }
        // The four lanes of a column add up.
#pragma unroll
        for (int half = 2; half >= 1; half >>= 1) {
          const bool up = (g & half) != 0;
#pragma unroll
          for (int j = 0; j < half; ++j) {
            const float2 send = up ? dw[j] : dw[j + half], keep = up ? dw[j + half] : dw[j];
            dw[j] = make_float2(keep.x + __shfl_xor_sync(0xFFFFFFFFu, send.x, 8 * half),
                                keep.y + __shfl_xor_sync(0xFFFFFFFFu, send.y, 8 * half));
          }
        }
        dweight = __fadd2_rn(dweight, dw[0]);
      }
      if constexpr (kHeld) {
        if (p.has_second) {
#pragma unroll
          for (int i = 0; i < 8; ++i) add_dsum(i, v[i]);
        }
        __syncwarp();
        if (ok && lane == 0 && panel + clusters < panels) load(panel + clusters);
        __syncwarp();
      }
    }
    rstd_next = load_rstd(panel + clusters);
    dead = sums_send<kWithheld>(sums, fold_rows(s, lane), dead, warp, lane, p.warps, crank, csize, k);
    const float total = sums_receive(sums, dead, lane, csize, k, p);
    const float mean = -rstd * (total / static_cast<float>(p.cols));
    if (!active) continue;
    [[maybe_unused]] float2 w[4];
    if constexpr (!kHeld) lane_weights(p, c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = __shfl_sync(0xFFFFFFFFu, rstd * mean, 8 * g + i);
      const float2 m2 = make_float2(m, m);
      if constexpr (!kHeld) {
        const float r = __shfl_sync(0xFFFFFFFFu, rstd, 8 * g + i);
        const float2 r2 = make_float2(r, r);
        unit_row_bf16(stage, 8 * g + i, q, v[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(__fmul2_rn(v[i][j], r2), w[j]);
        if (p.has_second) add_dsum(i, v[i]);
      }
      float2 h[4];
      unit_row<kF32>(stage + 4096, 8 * g + i, q, h);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = __ffma2_rn(h[j], m2, v[i][j]);
    }
    __syncwarp();
    if (ok && lane == 0 && panel + clusters < panels) {
      if constexpr (!kHeld) load(panel + clusters);
      load_sum(panel + clusters);
    }
    __syncwarp();
    if (p.out && c < p.cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * g + i < rows) store_row<kF32>(p.out, static_cast<int64_t>(row0 + 8 * g + i) * p.ld_out + c, v[i]);
    }
    if constexpr (kRow || kCol) store_unit<kRow, kCol>(v, p.q, lane, row0, rows, c0, p.cols, row0);
  }
  if (active && p.partial && c < p.cols) *reinterpret_cast<float2*>(p.partial + static_cast<int64_t>(cluster) * p.cols + c + 2 * g) = dweight;
  if (active && !ok && lane == 0) mbar_wait(bar, static_cast<uint32_t>(failed & 1), p.timeout_ns);
  __syncwarp();
  cluster_sync();  // no CTA leaves while another may still write to it
}

using Kernel = void (*)(const AddNormArgs);

template <bool kF32>
Kernel forward_kernel(bool row, bool col) {
  if (row && col) return add_norm_kernel<kF32, true, true>;
  if (row) return add_norm_kernel<kF32, true, false>;
  if (col) return add_norm_kernel<kF32, false, true>;
  return add_norm_kernel<kF32, false, false>;
}

template <bool kF32, int kThreads>
Kernel backward_kernel(bool row, bool col) {
  if (row && col) return add_norm_backward_kernel<kF32, true, true, kThreads>;
  if (row) return add_norm_backward_kernel<kF32, true, false, kThreads>;
  if (col) return add_norm_backward_kernel<kF32, false, true, kThreads>;
  return add_norm_backward_kernel<kF32, false, false, kThreads>;
}

// The backward kernel that holds its values gets 255 registers a thread up to 8 warps,
// 168 up to 12 (a few spilled); the other one 128.
template <bool kF32>
Kernel backward_kernel(bool row, bool col, bool held, int warps) {
  return !held        ? backward_kernel<kF32, 512>(row, col)
         : warps <= 8 ? backward_kernel<kF32, 256>(row, col)
                      : backward_kernel<kF32, 384>(row, col);
}

// Their variants for the self test, both copies.
template <bool kF32>
Kernel withheld_kernel(bool backward, bool held, int warps) {
  return !backward    ? add_norm_kernel<kF32, true, true, true>
         : !held      ? add_norm_backward_kernel<kF32, true, true, 512, true>
         : warps <= 8 ? add_norm_backward_kernel<kF32, true, true, 256, true>
                      : add_norm_backward_kernel<kF32, true, true, 384, true>;
}

// How a width is split: CTAs of a cluster, warps of a CTA; how many such clusters
// the GPU holds at once and CTAs an SM.
struct Split {
  int csize, warps, held, per_sm;
  bool holds;   // backward: the values stay in registers over the exchange
  bool direct;  // backward: dsum not through shared memory
  size_t smem;
  Kernel kern;
};

// Asks the runtime once for each kernel and shape on a device. held = 0: it does not fit.
cudaError_t occupancy(Split& s) {
  struct Entry {
    Kernel kern;
    int dev, csize, warps, held, per_sm;
    size_t smem;
  };
  static std::mutex mu;
  static std::vector<Entry> seen;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (const Entry& x : seen) {
    if (x.kern == s.kern && x.dev == dev && x.csize == s.csize && x.warps == s.warps && x.smem == s.smem) {
      s.held = x.held;
      s.per_sm = x.per_sm;
      return cudaSuccess;
    }
  }
  // A kernel's limit is the largest that one of its shapes can need.
  e = cudaFuncSetAttribute(s.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(s.kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.csize));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * s.warps));
  cfg.dynamicSmemBytes = s.smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(s.csize), 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  s.held = s.per_sm = 0;
  if (cudaOccupancyMaxActiveClusters(&s.held, s.kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    s.held = 0;
  }
  if (s.held > 0) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&s.per_sm, s.kern, 32 * s.warps, s.smem);
  if (e == cudaSuccess) seen.push_back(Entry{s.kern, dev, s.csize, s.warps, s.held, s.per_sm, s.smem});
  return e;
}

// One way to split the width; false where it cannot be.
bool split_of(const AddNormLaunch& L, int csize, bool held, Split* s) {
  const int64_t units = (L.cols + kUnitCols - 1) / kUnitCols;
  const bool row = L.row_data != nullptr, col = L.col_data != nullptr, f32 = L.stream_f32;
  *s = {};
  s->csize = csize;
  s->holds = held;
  s->warps = static_cast<int>((units + csize - 1) / csize);
  if (s->warps > kMaxWarps || (held && s->warps > 12)) return false;
  uint32_t stage = 4096 + unit_box_bytes(f32);
  if (L.backward && L.third) {
    // With an FP32 stream a whole stage is 22 KB a warp. Eight warps have one; nine (8193 to
    // 9216 columns) would find room but read dsum themselves as more do: 4096 x 9216 takes
    // 253 us, 36% of the copy rate, where 8192 x 8192 has 76%.
    s->direct = f32 && s->warps > 8;
    if (!s->direct) stage += unit_box_bytes(f32);
  }
  s->smem = 1024 + static_cast<size_t>(s->warps) * stage + sums_bytes(csize, s->warps);
  s->kern = !L.backward ? (f32 ? forward_kernel<true>(row, col) : forward_kernel<false>(row, col))
                        : (f32 ? backward_kernel<true>(row, col, held, s->warps) : backward_kernel<false>(row, col, held, s->warps));
  return true;
}

// The split with the least estimated time. A cluster takes one panel a round; a round
// takes a fixed time (the exchange; less where a second CTA of the SM works meanwhile)
// and one in proportion to the SM's warps. Measured on GB300, us: forward 1.2 (0.7) +
// 0.37 a warp, backward 1.0 + 0.40 with its values held over the exchange, else 2.0 (0.3)
// + 0.48. What that decides (BF16 stream, both copies): forward 8192 x 5120 clusters of 5
// CTAs x 16 warps 65.7 us, of 8 x 10 82, 16 x 5 72; 8192 x 7168 8 x 14 100, 7 x 16 107,
// 16 x 7 104 (FP32 stream: 154, 170, 146); backward, held and not: 16384 x 2048 4 x 8 70.1
// and 67.4, 2 x 16 - and 72.7; 8192 x 4096 6 x 11 74.3 and 94.1, 8 x 8 79.5 and 69.8; 8192 x
// 7168 16 x 7 154.7 and 133.9; 32768 x 1408 2 x 11 85.8 and 104.8, 6 x 4 96.3 and 86.7; 4096 x
// 12288 16 x 12 119 and 146. With an FP32 stream the values are held wherever they can
// be (8192 x 7168: 197 us, and 308): its stages leave room for 9 warps of an SM. Clusters of
// ten and twelve leave fewer of a GPC's SMs over than those of eight at some widths:
// forward 8192 x 5120 10 x 8 60.3 us, 8192 x 6144 with an FP32 stream 12 x 8 113.8 (16 x 6
// 129.4); backward 8192 x 5120 10 x 8 84.7 (5 x 16 98.3), FP32 stream 124 (16 x 5 174), 8192 x
// 7168 10 x 12 125. Of nine, eleven and thirteen to fifteen one alone was the fastest at one
// width, nine (forward 8192 x 8192: 105.9, eight 108.0); they are left out.
mx_status choose(const AddNormLaunch& L, Split* out) {
  const int64_t panels = (L.rows + 31) / 32;
  double best = 0.0;
  out->held = 0;
  for (int csize : {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, kMaxCluster}) {
    for (const bool held : {true, false}) {
      Split s;
      if (held && !L.backward) continue;
      if (!split_of(L, csize, held, &s) || (s.warps < 4 && out->held > 0)) continue;
      if (L.backward && !held && L.stream_f32 && s.warps <= 12) continue;
      const cudaError_t e = occupancy(s);
      if (e != cudaSuccess) return cuda_status(e, "add_norm occupancy");
      if (s.held < 1) continue;
      const int64_t clusters = std::min<int64_t>(s.held, kMaxParts);
      const bool two = s.per_sm > 1;
      const double fixed = !L.backward ? (two ? 0.7 : 1.2) : held ? 1.0 : (two ? 0.3 : 2.0);
      // fewer panels than clusters: an SM has one CTA
      const int per_sm = panels * csize <= sm_count() ? 1 : std::max(1, s.per_sm);
      double t = static_cast<double>((panels + clusters - 1) / clusters) *
                 (fixed + (!L.backward ? 0.37 : held ? 0.40 : 0.48) * s.warps * per_sm);
      if (s.direct) t *= 2.0;  // 8192 x 7168: 394 us with dsum read by the lanes, 197 through shared memory
      if (out->held == 0 || t < best) {
        best = t;
        *out = s;
      }
    }
  }
  if (out->held > 0) return MX_OK;
  return cuda_status(cudaErrorInvalidConfiguration, "add_norm clusters");
}

}  // namespace

mx_status make_unit_map(CUtensorMap* map, bool f32, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static EncodeTiledFn enc = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      enc = reinterpret_cast<EncodeTiledFn>(f);
  });
  if (!enc) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return MX_ERR_CUDA;
  }
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {f32 ? 32u : 64u, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                         const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled (32 x 64 units) failed (%d)", static_cast<int>(r));
    return MX_ERR_CUDA;
  }
  return MX_OK;
}

size_t add_norm_backward_workspace(int64_t rows, int64_t cols) {
  return static_cast<size_t>(std::min<int64_t>((rows + 31) / 32, kMaxParts)) * static_cast<size_t>(cols) * sizeof(float);
}

mx_status launch_add_norm(const AddNormLaunch& L, cudaStream_t s) {
  // A model's layers call with the same sizes over and over: the thread's last split of
  // each direction and stream type stands while what it was chosen by does.
  struct Chosen {
    int64_t rows, cols;
    int dev, flags;
    Split split;
  };
  static thread_local Chosen last[4] = {};
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
  const int flags = 1 | (L.row_data ? 2 : 0) | (L.col_data ? 4 : 0) | (L.third ? 8 : 0);
  Chosen& ch = last[(L.backward ? 2 : 0) + (L.stream_f32 ? 1 : 0)];
  mx_status st = MX_OK;
  if (ch.rows != L.rows || ch.cols != L.cols || ch.dev != dev || ch.flags != flags) {
    Split found;
    st = choose(L, &found);
    if (st != MX_OK) return st;
    ch = Chosen{L.rows, L.cols, dev, flags, found};
  }
  Split sp = ch.split;
  const WaitTest test = take_wait_test();
  if (test.sums() && L.row_data && L.col_data) {
    sp.kern = L.stream_f32 ? withheld_kernel<true>(L.backward, sp.holds, sp.warps) : withheld_kernel<false>(L.backward, sp.holds, sp.warps);
    if (const cudaError_t e = occupancy(sp); e != cudaSuccess || sp.held < 1)
      return cuda_status(e != cudaSuccess ? e : cudaErrorInvalidConfiguration, "add_norm self test");
  }
  AddNormArgs a = {};
  a.weight = L.weight;
  a.weight_f32 = L.param_dtype == MX_F32;
  a.weight_vec = (reinterpret_cast<uintptr_t>(L.weight) & 15u) == 0;
  a.rows = L.rows;
  a.cols = L.cols;
  a.eps = L.eps;
  a.warps = sp.warps;
  a.dev_status = L.dev_status;
  a.timeout_ns = test.limit();
  a.out = L.out;
  a.ld_out = L.ld_out;
  a.y = static_cast<__nv_bfloat16*>(L.y);
  a.ldy = L.ldy;
  a.rstd = L.rstd;
  a.rstd_in = L.rstd;
  a.q = CopyOut{static_cast<uint8_t*>(L.row_data), static_cast<uint8_t*>(L.row_scale), static_cast<uint8_t*>(L.col_data),
                static_cast<uint8_t*>(L.col_scale), L.cols, (L.cols + 127) / 128, L.rows, (L.rows + 127) / 128};
  st = make_unit_map(&a.a, false, L.first, L.cols, L.rows, L.ld_first, test.stages() ? kUnitRows / 2 : kUnitRows);
  if (st == MX_OK && L.second) st = make_unit_map(&a.b, L.stream_f32, L.second, L.cols, L.rows, L.ld_second);
  if (st == MX_OK && L.third && !sp.direct) st = make_unit_map(&a.c, L.stream_f32, L.third, L.cols, L.rows, L.ld_third);
  if (st != MX_OK) return st;
  if (L.backward) {
    a.has_second = L.third ? (sp.direct ? 2 : 1) : 0;
    a.direct = L.third;
    a.ld_direct = L.ld_third;
    a.partial = L.dweight ? static_cast<float*>(L.ws) : nullptr;
  } else {
    a.has_second = L.second != nullptr;
  }
  const int clusters = static_cast<int>(std::min<int64_t>({(L.rows + 31) / 32, sp.held, kMaxParts}));
  st = cuda_status(launch_kernel(sp.kern, static_cast<unsigned>(clusters * sp.csize), static_cast<unsigned>(32 * sp.warps),
                                 sp.smem, s, static_cast<unsigned>(sp.csize), a),
                   L.backward ? "mx_add_norm_backward launch" : "mx_add_norm_quantize launch");
  if (st != MX_OK || !L.dweight) return st;
  // A next kernel that is placed while the sums' CTAs hold some SMs' registers comes out
  // lopsided, for all of its time if it is one of clusters such as this: 16384 x 2048, call
  // after call, 68 to 88 us, and 66 behind the sums.
  return launch_column_reduce(a.partial, clusters, L.cols, 0, L.dweight, nullptr, s, true);
}

}  // namespace mx
