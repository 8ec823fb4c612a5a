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
// and stays in their registers in FP32 from the load to the stores. Per panel the
// warps exchange one sum for each row: warps of a CTA through shared memory, CTAs
// through each other's shared memory and a cluster barrier, added in a fixed order.
// Each warp's part of the next panel is on its way into shared memory (TMA, one
// stage per warp, its own mbarrier) as soon as the present one is in registers.
//
// A wait that runs out leaves MX_ERR_TIMEOUT, and NaN in the values it was for; the
// warp loads nothing more, but takes part in every barrier.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "mx_block.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kMaxCluster = 16;   // CTAs (above 8: opt-in)
constexpr int kMaxWarps = 16;     // of a CTA
constexpr int kMaxParts = 608;    // clusters of a launch (partial rows of dweight)

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
  float (*part)[32];            // [warps][32]
  volatile uint64_t (*all)[32]; // [2 * CTAs][32]
};

// Both in dynamic shared memory, behind the stages.
constexpr size_t sums_bytes(int csize, int warps) { return static_cast<size_t>(csize) * 2 * 32 * 8 + static_cast<size_t>(warps) * 32 * 4; }

__device__ __forceinline__ RowSums sums_at(uint8_t* at, uint32_t csize) {
  return RowSums{reinterpret_cast<float(*)[32]>(at + csize * 2 * 32 * 8), reinterpret_cast<volatile uint64_t(*)[32]>(at)};
}

// `dead`: a wait of this warp has run out. Once one of the CTA's has, the CTA sends
// nothing more (its panels come out as NaN, and the others' waits run out too):
// returns true then.
__device__ __forceinline__ bool sums_send(const RowSums& s, float mine, bool dead, int warp, int lane, int warps, uint32_t crank,
                                          uint32_t csize, int k) {
  s.part[warp][lane] = mine;
  if (__syncthreads_or(dead)) return true;
  if (warp == 0) {
    float t = 0.0f;
    for (int w = 0; w < warps; ++w) t += s.part[w][lane];
    const uint64_t word = (static_cast<uint64_t>(static_cast<uint32_t>(k) + 1u) << 32) | __float_as_uint(t);
    const uint32_t at = smem_u32(const_cast<uint64_t*>(&s.all[(k & 1) * csize + crank][lane]));
    for (uint32_t r = 0; r < csize; ++r) st_cluster_u64(mapa_shared(at, r), word);
  }
  return false;
}

// After sums_send of panel k; NaN, and dead, where the wait runs out.
__device__ __forceinline__ float sums_receive(const RowSums& s, bool& dead, int lane, uint32_t csize, int k,
                                              const AddNormArgs& p) {
  if (dead) return __int_as_float(0x7FFFFFFF);
  const uint32_t number = static_cast<uint32_t>(k) + 1u;
  float t = 0.0f;
  bool there = true;
  for (uint32_t r = 0; r < csize; ++r) {
    volatile uint64_t* at = &s.all[(k & 1) * csize + r][lane];
    uint64_t word = *at;
    if (static_cast<uint32_t>(word >> 32) != number) {
      const uint64_t t0 = global_timer_ns();
      do {
#pragma unroll 1
        for (int i = 0; i < 64 && static_cast<uint32_t>(word >> 32) != number; ++i) word = *at;
        there = static_cast<uint32_t>(word >> 32) == number;
      } while (!there && global_timer_ns() - t0 <= p.timeout_ns);
      if (!there) break;
    }
    t += __uint_as_float(static_cast<uint32_t>(word));
  }
  if (!there && p.dev_status) atomicExch(p.dev_status, static_cast<int>(MX_ERR_TIMEOUT));
  dead = !__all_sync(0xFFFFFFFFu, there);
  return dead ? __int_as_float(0x7FFFFFFF) : t;
}

__device__ __forceinline__ void lane_weights(const AddNormArgs& p, int64_t c, float2 (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = make_float2(c < p.cols ? 1.0f : 0.0f, c < p.cols ? 1.0f : 0.0f);
  if (!p.weight || c >= p.cols) return;
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
__device__ __forceinline__ void load_box(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int64_t c0, int64_t row0) {
  tma_load_2d(dst, map, bar, static_cast<int32_t>(c0), static_cast<int32_t>(row0));
  if constexpr (kF32) tma_load_2d(dst + kF32Box, map, bar, static_cast<int32_t>(c0 + 32), static_cast<int32_t>(row0));
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
template <bool kF32, bool kRow, bool kCol, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) add_norm_kernel(const __grid_constant__ AddNormArgs p) {
  constexpr uint32_t kStage = 4096 + unit_box_bytes(kF32);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_bar[kMaxWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 7, g = lane >> 3;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();
  const int64_t cluster = blockIdx.x / csize, clusters = gridDim.x / csize;
  const int64_t panels = (p.rows + 31) >> 5;
  const int64_t c0 = (static_cast<int64_t>(crank) * p.warps + warp) * kUnitCols;
  const int64_t c = c0 + 8 * q;
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
  for (uint32_t i = warp; i < 2 * csize; i += p.warps) sums.all[i][lane] = 0;
  pdl_launch_dependents();
  cluster_sync();  // every CTA of the cluster runs before one writes to it
  pdl_wait();

  auto load = [&](int64_t panel) {
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
  for (int64_t panel = cluster; panel < panels; panel += clusters, ++k) {
    const int64_t row0 = panel * 32;
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
    dead = sums_send(sums, fold_rows(s, lane), dead, warp, lane, p.warps, crank, csize, k);
    if (active && p.out && c < p.cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * g + i < rows) store_row<kF32>(p.out, (row0 + 8 * g + i) * p.ld_out + c, v[i]);
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
        if (8 * g + i < rows) store_row<false>(p.y, (row0 + 8 * g + i) * p.ldy + c, v[i]);
    }
    store_unit<kRow, kCol>(v, p.q, lane, row0, rows, c0, p.cols, row0);
  }
  // A warp that gave up has one load on its way at most: its stage's.
  if (active && !ok && lane == 0) mbar_wait(bar, static_cast<uint32_t>(failed & 1), p.timeout_ns);
  __syncwarp();
  cluster_sync();  // no CTA leaves while another may still write to it
}

template <bool kF32, bool kRow, bool kCol, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) add_norm_backward_kernel(const __grid_constant__ AddNormArgs p) {
  constexpr uint32_t kStream = unit_box_bytes(kF32);
  const uint32_t streams = p.has_second == 1 ? 2 : 1, stage_bytes = 4096 + streams * kStream;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_bar[kMaxWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 7, g = lane >> 3;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();
  const int64_t cluster = blockIdx.x / csize, clusters = gridDim.x / csize;
  const int64_t panels = (p.rows + 31) >> 5;
  const int64_t c0 = (static_cast<int64_t>(crank) * p.warps + warp) * kUnitCols;
  const int64_t c = c0 + 8 * q;
  const bool active = c0 < p.cols;
  uint8_t* stage = smem + warp * stage_bytes;
  uint64_t* bar = &s_bar[warp];
  const RowSums sums = sums_at(smem + p.warps * stage_bytes, csize);

  if (lane == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  for (uint32_t i = warp; i < 2 * csize; i += p.warps) sums.all[i][lane] = 0;
  pdl_launch_dependents();
  cluster_sync();  // every CTA of the cluster runs before one writes to it
  pdl_wait();

  auto load = [&](int64_t panel) {
    mbar_arrive_expect_tx(bar, 4096 + streams * (kF32 ? 8192 : 4096));
    load_box<false>(stage, &p.a, bar, c0, panel * 32);
    load_box<kF32>(stage + 4096, &p.b, bar, c0, panel * 32);
    if (p.has_second == 1) load_box<kF32>(stage + 4096 + kStream, &p.c, bar, c0, panel * 32);
  };
  if (active && lane == 0 && cluster < panels) load(cluster);
  float2 w[4], dw[4];
  lane_weights(p, c, w);
#pragma unroll
  for (int j = 0; j < 4; ++j) dw[j] = make_float2(0.0f, 0.0f);
  {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, n = static_cast<int64_t>(gridDim.x) * blockDim.x;
    if (kRow) zero_scale_padding(p.q.row_scale, p.rows, p.cols >> 5, p.q.row_ka, id, n);
    if (kCol) zero_scale_padding(p.q.col_scale, p.cols, p.rows >> 5, p.q.col_ka, id, n);
  }

  bool ok = true, dead = false;
  int k = 0, failed = 0;
  for (int64_t panel = cluster; panel < panels; panel += clusters, ++k) {
    const int64_t row0 = panel * 32;
    const int rows = static_cast<int>(min64(32, p.rows - row0));
    const float rstd = lane < rows ? p.rstd_in[row0 + lane] : 0.0f;
    float2 v[8][4], h[8][4];  // dsum + rstd g; h
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (active) {
      if (ok) {
        ok = __all_sync(0xFFFFFFFFu, stage_wait(bar, k & 1, p));
        failed = k;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float r = __shfl_sync(0xFFFFFFFFu, rstd, 8 * g + i);
        const float2 r2 = make_float2(r, r);
        float2 dy[4], t = make_float2(0.0f, 0.0f);
        if (ok) {
          unit_row_bf16(stage, 8 * g + i, q, dy);
          unit_row<kF32>(stage + 4096, 8 * g + i, q, h[i]);
          if (p.has_second == 1) {
            unit_row<kF32>(stage + 4096 + kStream, 8 * g + i, q, v[i]);
          } else if (p.has_second == 2 && 8 * g + i < rows && c < p.cols) {
            load_row<kF32>(p.direct, (row0 + 8 * g + i) * p.ld_direct + c, v[i]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = make_float2(0.0f, 0.0f);
          }
        } else {
          fill_nan(dy);
          fill_nan(h[i]);
          fill_nan(v[i]);
        }
        if (8 * g + i >= rows) {  // zeros from the load; rstd 0
#pragma unroll
          for (int j = 0; j < 4; ++j) dy[j] = h[i][j] = v[i][j] = make_float2(0.0f, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i][j] = __fmul2_rn(h[i][j], r2);
          dw[j] = __ffma2_rn(dy[j], h[i][j], dw[j]);
          dy[j] = __fmul2_rn(dy[j], w[j]);
          t = __ffma2_rn(dy[j], h[i][j], t);
          v[i][j] = __ffma2_rn(dy[j], r2, v[i][j]);
        }
        s[i] = t.x + t.y;
      }
      __syncwarp();
      if (ok && lane == 0 && panel + clusters < panels) load(panel + clusters);
      __syncwarp();
    }
    dead = sums_send(sums, fold_rows(s, lane), dead, warp, lane, p.warps, crank, csize, k);
    const float total = sums_receive(sums, dead, lane, csize, k, p);
    const float mean = -rstd * (total / static_cast<float>(p.cols));
    if (!active) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = __shfl_sync(0xFFFFFFFFu, mean, 8 * g + i);
      const float2 m2 = make_float2(m, m);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = __ffma2_rn(h[i][j], m2, v[i][j]);
      if (p.out && c < p.cols && 8 * g + i < rows) store_row<kF32>(p.out, (row0 + 8 * g + i) * p.ld_out + c, v[i]);
    }
    if constexpr (kRow || kCol) store_unit<kRow, kCol>(v, p.q, lane, row0, rows, c0, p.cols, row0);
  }
  if (active && p.partial) {
    // The four lanes of a column add up: lane 8 g + q ends with columns 8 q + 2 g and + 1.
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
    if (c < p.cols) *reinterpret_cast<float2*>(p.partial + cluster * p.cols + c + 2 * g) = dw[0];
  }
  if (active && !ok && lane == 0) mbar_wait(bar, static_cast<uint32_t>(failed & 1), p.timeout_ns);
  __syncwarp();
  cluster_sync();  // no CTA leaves while another may still write to it
}

// How a width is split: CTAs of a cluster and warps of a CTA.
struct Split {
  int csize, warps;
};

Split split_of(int64_t cols, int max_warps) {
  const int64_t units = (cols + kUnitCols - 1) / kUnitCols;
  Split s{1, 1};
  while (s.csize < kMaxCluster && static_cast<int64_t>(s.csize) * max_warps < units) s.csize *= 2;
  s.warps = static_cast<int>((units + s.csize - 1) / s.csize);
  return s;
}

using Kernel = void (*)(const AddNormArgs);

template <int kThreads, bool kBackward, bool kF32>
Kernel kernel_of(bool row, bool col) {
  if constexpr (kBackward) {
    if (row && col) return add_norm_backward_kernel<kF32, true, true, kThreads>;
    if (row) return add_norm_backward_kernel<kF32, true, false, kThreads>;
    if (col) return add_norm_backward_kernel<kF32, false, true, kThreads>;
    return add_norm_backward_kernel<kF32, false, false, kThreads>;
  } else {
    if (row && col) return add_norm_kernel<kF32, true, true, kThreads>;
    if (row) return add_norm_kernel<kF32, true, false, kThreads>;
    if (col) return add_norm_kernel<kF32, false, true, kThreads>;
    return add_norm_kernel<kF32, false, false, kThreads>;
  }
}

mx_status launch(Kernel kern, AddNormArgs& a, const Split& sp, size_t smem, cudaStream_t s, int* clusters_out) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess && sp.csize > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(add_norm)");
  // As many clusters as the GPU holds at once (each then walks its panels).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sp.csize));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * sp.warps));
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(sp.csize), 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int held = 0;
  e = cudaOccupancyMaxActiveClusters(&held, kern, &cfg);
  if (e != cudaSuccess || held < 1) return cuda_status(e == cudaSuccess ? cudaErrorInvalidConfiguration : e, "add_norm clusters");
  const int64_t panels = (a.rows + 31) / 32;
  const int clusters = static_cast<int>(std::min<int64_t>({panels, held, kMaxParts}));
  a.warps = sp.warps;
  a.timeout_ns = wait_timeout_ns();
  *clusters_out = clusters;
  return cuda_status(launch_kernel(kern, static_cast<unsigned>(clusters * sp.csize), static_cast<unsigned>(32 * sp.warps), smem,
                                   s, static_cast<unsigned>(sp.csize), a),
                     "add_norm launch");
}

}  // namespace

mx_status make_unit_map(CUtensorMap* map, bool f32, const void* base, int64_t cols, int64_t rows, int64_t ld) {
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
  const cuuint32_t box[2] = {f32 ? 32u : 64u, static_cast<cuuint32_t>(kUnitRows)};
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
  AddNormArgs a = {};
  a.weight = L.weight;
  a.weight_f32 = L.param_dtype == MX_F32;
  a.rows = L.rows;
  a.cols = L.cols;
  a.eps = L.eps;
  a.dev_status = L.dev_status;
  a.out = L.out;
  a.ld_out = L.ld_out;
  a.y = static_cast<__nv_bfloat16*>(L.y);
  a.ldy = L.ldy;
  a.rstd = L.rstd;
  a.rstd_in = L.rstd;
  a.q = CopyOut{static_cast<uint8_t*>(L.row_data), static_cast<uint8_t*>(L.row_scale), static_cast<uint8_t*>(L.col_data),
                static_cast<uint8_t*>(L.col_scale), L.cols, (L.cols + 127) / 128, L.rows, (L.rows + 127) / 128};
  const bool f32 = L.stream_f32, row = L.row_data != nullptr, col = L.col_data != nullptr;
  mx_status st = make_unit_map(&a.a, false, L.first, L.cols, L.rows, L.ld_first);
  if (st != MX_OK) return st;
  int clusters = 0;
  const Split sp = split_of(L.cols, L.cols > 8192 ? 16 : 8);
  if (!L.backward) {
    a.has_second = L.second != nullptr;
    if (L.second) st = make_unit_map(&a.b, f32, L.second, L.cols, L.rows, L.ld_second);
    if (st != MX_OK) return st;
    const size_t smem = 1024 + static_cast<size_t>(sp.warps) * (4096 + unit_box_bytes(f32)) + sums_bytes(sp.csize, sp.warps);
    const Kernel kern = sp.warps > 8 ? (f32 ? kernel_of<512, false, true>(row, col) : kernel_of<512, false, false>(row, col))
                                     : (f32 ? kernel_of<256, false, true>(row, col) : kernel_of<256, false, false>(row, col));
    return launch(kern, a, sp, smem, s, &clusters);
  }
  a.has_second = L.third != nullptr;
  st = make_unit_map(&a.b, f32, L.second, L.cols, L.rows, L.ld_second);
  if (st == MX_OK && L.third) st = make_unit_map(&a.c, f32, L.third, L.cols, L.rows, L.ld_third);
  if (st != MX_OK) return st;
  a.partial = L.dweight ? static_cast<float*>(L.ws) : nullptr;
  // With an FP32 stream a whole stage is 22 KB a warp; where a CTA's warps do not
  // find room for that (above 9216 columns), dsum does not come through it.
  if (a.has_second && f32 && sp.warps > 9) {
    a.has_second = 2;
    a.direct = L.third;
    a.ld_direct = L.ld_third;
  }
  const size_t smem = 1024 + static_cast<size_t>(sp.warps) * (4096 + (a.has_second == 1 ? 2 : 1) * unit_box_bytes(f32)) +
                      sums_bytes(sp.csize, sp.warps);
  const Kernel kern = sp.warps > 8 ? (f32 ? kernel_of<512, true, true>(row, col) : kernel_of<512, true, false>(row, col))
                                   : (f32 ? kernel_of<256, true, true>(row, col) : kernel_of<256, true, false>(row, col));
  st = launch(kern, a, sp, smem, s, &clusters);
  if (st != MX_OK || !L.dweight) return st;
  return launch_column_reduce(a.partial, clusters, L.cols, 0, L.dweight, nullptr, s);
}

}  // namespace mx
