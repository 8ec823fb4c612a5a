// mx_gated.cu - between the two products of a gated feed-forward block, on
// gate_up = [gate | up] in BF16, [rows, 2F]:
//
//   forward:   h = act(gate) up                            -> MX copies of h
//   backward:  dgate = dh up act'(gate), dup = dh act(gate) -> MX copies of [dgate | dup]
//
// dense, or with the column copy in the experts' segments (padded with zero codes
// to a multiple of 128 rows, as mx_quantize's). The values go from FP32 registers
// into the blocks and are never written in BF16: 6.06 bytes per value of F forward,
// 10.13 backward, which HBM bounds; through a BF16 tensor it would be 10.06 and
// 18.13.
//
// Four warps take a tile of 128 rows x 64 columns of F, 32 x 64 each (mx_block.cuh): a
// warp's next unit is on its way into shared memory (TMA, its own mbarrier) while it
// works on the present one. The row copy goes out from the registers, the column copy
// through shared memory, 128 bytes a column at a time. The activation is computed once
// for both copies and both gradients.
//
// Measured, both copies, SiLU (of 6787 GB/s copied): forward 49152 x 1408, 64 experts
// 71 us (87%), 8192 x 10944 89 us (90%); backward 117 us (88%) and 144 us (93%).

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mx_act.cuh"
#include "mx_block.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kTile = 128;  // rows of a CTA's tile

// Units side by side in a CTA's tile, four warps each, and CTAs of an SM. Three shapes:
// forward 1 x 3 (12 warps of 168 registers) or 2 x 2 (16 of 128), backward 2 x 1 or 1 x 2 (8
// of 219). Dense matrices and row copies alone take the first of each, column copies of
// groups the second; us of first and second:
//   dense    forward   8192 x 10944: 88.7, 96.4   49152 x 1408: 69.8, 69.9   512 x 1408: 3.9, 4.3
//            backward  8192 x 10944: 144, 156     49152 x 1408: 113, 111
//   groups   forward   49152 x 1408, 64: 76.0, 70.6  256: 91.2, 84.4   16384 x 4096, 8: 71.2, 69.2
//            backward  49152 x 1408, 64: 123, 117    256: 151, 143     16384 x 4096, 8: 116, 111
//                      8192 x 10944, 4: 151, 145 (forward 92.5, 101: there the rule costs 9%)
__host__ __device__ constexpr int units_across(bool backward, bool second) { return backward != second ? 2 : 1; }
__host__ __device__ constexpr int ctas_per_sm(bool backward, bool second) { return backward ? (second ? 2 : 1) : (second ? 2 : 3); }

struct GatedArgs {
  CUtensorMap dh, gate, up;
  CopyOut q;
  int64_t rows, f;
  int64_t tiles_c;         // tiles along F
  int64_t tiles_r;         // tiles along the rows (dense)
  const int64_t* offsets;
  int32_t n_groups;
  int64_t capacity;
  int* dev_status;
  uint64_t timeout_ns;
};

// A CTA's tiles, one after the other: row tile, column tile, and the group that the
// row tile is in. They go along F first, `step` tiles at a time.
struct Walk {
  int32_t rt, ct, group;
  int32_t step_r, step_c;  // the step in whole row tiles, and the rest of it
};

// A warp's unit of a tile.
struct Unit {
  int64_t kpos;
  int32_t row0, c0;
  int32_t rows;  // that exist, <= 0: none
};

template <int kAcross>
__device__ __forceinline__ Unit unit_of(const GatedArgs& p, const Walk& w, int warp, const int32_t* off, const int32_t* tile) {
  Unit u;
  const int32_t r = (warp & 3) * kUnitRows;
  u.c0 = (w.ct * kAcross + (warp >> 2)) * kUnitCols;
  u.kpos = static_cast<int64_t>(w.rt) * kTile + r;
  if (off) {
    const int32_t in = (w.rt - tile[w.group]) * kTile + r;  // row within the group
    u.row0 = off[w.group] + in;
    u.rows = min(kUnitRows, off[w.group + 1] - off[w.group] - in);
  } else {
    u.row0 = static_cast<int32_t>(u.kpos);
    u.rows = static_cast<int32_t>(min64(kUnitRows, p.rows - u.kpos));
  }
  if (u.c0 >= p.f) u.rows = 0;
  return u;
}

// The group with tiles that row tile w.rt is in, from w.group on.
__device__ __forceinline__ void find_group(Walk& w, const int32_t* tile) {
  while (tile[w.group + 1] <= w.rt) ++w.group;
}

// Offsets of the groups, and their first tiles, into shared memory; returns how
// many tiles they have, or -1 (status recorded) if they or the capacity are wrong.
__device__ int32_t setup_groups(const GatedArgs& p, bool col, int32_t* off, int32_t* tile, int32_t* flag) {
  const int tid = threadIdx.x, E = p.n_groups;
  if (tid == 0) *flag = 0;
  __syncthreads();
  for (int e = tid; e <= E; e += blockDim.x) {
    const int64_t o = p.offsets[e];
    off[e] = static_cast<int32_t>(o);
    if (o < 0 || o > p.rows || (e == 0 && o != 0) || (e == E && o != p.rows) || (e > 0 && o < p.offsets[e - 1])) *flag = 1;
  }
  __syncthreads();
  if (*flag == 0 && tid < 32) {
    // Exclusive prefix of the groups' tiles, 32 groups a step.
    int32_t before = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + tid;
      int32_t n = e < E ? (off[e + 1] - off[e] + kTile - 1) / kTile : 0;
      const int32_t mine = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t t = __shfl_up_sync(0xFFFFFFFFu, n, d);
        if (tid >= d) n += t;
      }
      if (e < E) tile[e] = before + n - mine;
      before += __shfl_sync(0xFFFFFFFFu, n, 31);
    }
    if (tid == 0) {
      tile[E] = before;
      if (col && static_cast<int64_t>(before) * kTile > p.capacity) *flag = 1;
    }
  }
  __syncthreads();
  if (*flag) {
    if (tid == 0 && blockIdx.x == 0 && p.dev_status) atomicExch(p.dev_status, static_cast<int>(MX_ERR_DEVICE_CHECK));
    return -1;
  }
  return tile[E];
}

// The four warps of a unit's column.
__device__ __forceinline__ void column_sync(int column) { asm volatile("bar.sync %0, 128;" ::"r"(column + 1) : "memory"); }

template <int kAct, bool kBackward, bool kRow, bool kCol, bool kSecond>
__global__ void __launch_bounds__(128 * units_across(kBackward, kSecond), ctas_per_sm(kBackward, kSecond))
    gated_kernel(const __grid_constant__ GatedArgs p) {
  constexpr int kAcross = units_across(kBackward, kSecond), kWarps = 4 * kAcross;
  constexpr uint32_t kStage = kBackward ? 3 * 4096 : 2 * 4096;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_bar[kWarps];
  __shared__ int32_t s_off[MX_MAX_GROUPS + 1], s_tile[MX_MAX_GROUPS + 1], s_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 7, g = lane >> 3;
  uint8_t* stage = smem + warp * kStage;
  uint8_t* const stage0 = smem + kWarps * kStage + (warp >> 2) * 2 * kStagedBytes;  // two tiles of column copies
  uint8_t* staged = stage0;
  uint64_t* bar = &s_bar[warp];
  if (lane == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();

  int64_t tiles_r = p.tiles_r;
  const int32_t* off = nullptr;
  if (p.offsets) {
    tiles_r = setup_groups(p, kCol, s_off, s_tile, &s_flag);
    if (tiles_r < 0) return;
    off = s_off;
  }
  const int64_t width = kBackward ? 2 * p.f : p.f;
  {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, n = static_cast<int64_t>(gridDim.x) * blockDim.x;
    if (kRow) zero_scale_padding(p.q.row_scale, p.rows, width >> 5, p.q.row_ka, id, n);
    if (kCol) zero_scale_padding(p.q.col_scale, width, (off ? tiles_r * kTile : p.rows) >> 5, p.q.col_ka, id, n);
  }

  auto load = [&](const Unit& u) {
    mbar_arrive_expect_tx(bar, kStage);
    tma_load_2d(stage, &p.gate, bar, u.c0, u.row0);
    tma_load_2d(stage + 4096, &p.up, bar, u.c0, u.row0);
    if (kBackward) tma_load_2d(stage + 8192, &p.dh, bar, u.c0, u.row0);
  };

  // The warps of a CTA walk the same tiles; without a column copy they never wait for
  // one another, with one a unit's four meet once for each output.
  bool ok = true;
  uint32_t phase = 0;
  const int32_t tiles_c = static_cast<int32_t>(p.tiles_c), last_r = static_cast<int32_t>(tiles_r);
  Walk w;
  w.step_r = static_cast<int32_t>(gridDim.x) / tiles_c;
  w.step_c = static_cast<int32_t>(gridDim.x) % tiles_c;
  w.rt = static_cast<int32_t>(blockIdx.x) / tiles_c;
  w.ct = static_cast<int32_t>(blockIdx.x) % tiles_c;
  w.group = 0;
  if (w.rt >= last_r) return;
  if (off) find_group(w, s_tile);
  Unit u = unit_of<kAcross>(p, w, warp, off, s_tile);
  if (lane == 0 && u.rows > 0) load(u);
  __syncwarp();
  for (bool more = true; more;) {
    const Unit now = u;
    if (now.rows > 0 && ok) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase, p.timeout_ns));
      if (!ok) {
        // Nothing more is loaded; what is left comes out as NaN.
        if (lane == 0) {
          if (p.dev_status) atomicExch(p.dev_status, static_cast<int>(MX_ERR_TIMEOUT));
          mbar_wait(bar, phase, p.timeout_ns);
        }
        __syncwarp();
      }
      phase ^= 1;
    }
    float2 a[8][4];                   // h, or dgate
    [[maybe_unused]] float2 b[8][4];  // dup
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * g + i;
      float2 gate[4], up[4];
      unit_row_bf16(stage, r, q, gate);
      unit_row_bf16(stage + 4096, r, q, up);
      if constexpr (kBackward) {
        float2 dh[4];
        unit_row_bf16(stage + 8192, r, q, dh);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 value, slope;
          act_both<kAct>(gate[j], value, slope);
          a[i][j] = __fmul2_rn(__fmul2_rn(dh[j], up[j]), slope);
          b[i][j] = __fmul2_rn(dh[j], value);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) a[i][j] = __fmul2_rn(act_value<kAct>(gate[j]), up[j]);
      }
    }
    __syncwarp();
    // The next unit's loads into the same stage.
    w.rt += w.step_r;
    w.ct += w.step_c;
    if (w.ct >= tiles_c) {
      w.ct -= tiles_c;
      ++w.rt;
    }
    more = w.rt < last_r;
    if (more) {
      if (off) find_group(w, s_tile);
      u = unit_of<kAcross>(p, w, warp, off, s_tile);
      if (ok && lane == 0 && u.rows > 0) load(u);
      __syncwarp();
    }
    if (!ok || now.rows < kUnitRows) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool there = 8 * g + i < now.rows;
        const float fill = !ok && there ? __int_as_float(0x7FFFFFFF) : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!there || !ok) a[i][j] = make_float2(fill, fill);
          if constexpr (kBackward)
            if (!there || !ok) b[i][j] = make_float2(fill, fill);
        }
      }
    }
    const int64_t tile_k = now.kpos - (warp & 3) * kUnitRows, k_end = off ? INT64_MAX : p.rows;
    store_unit<kRow, kCol, true>(a, p.q, lane, now.row0, now.rows, now.c0, p.f, now.kpos, staged, warp & 3);
    if constexpr (kCol) {
      column_sync(warp >> 2);
      store_columns(staged, p.q, warp & 3, lane, now.c0, p.f, tile_k, k_end);
    }
    if constexpr (kBackward) {
      store_unit<kRow, kCol, true>(b, p.q, lane, now.row0, now.rows, now.c0 + p.f, 2 * p.f, now.kpos, staged + kStagedBytes,
                                   warp & 3);
      if constexpr (kCol) {
        column_sync(warp >> 2);
        store_columns(staged + kStagedBytes, p.q, warp & 3, lane, now.c0 + p.f, 2 * p.f, tile_k, k_end);
      }
    } else if (kCol) {
      staged = staged == stage0 ? stage0 + kStagedBytes : stage0;  // read while the next is written
    }
  }
}

using Kernel = void (*)(const GatedArgs);

template <int kAct, bool kBackward>
Kernel kernel_of(bool row, bool col, bool second) {
  if (row && col) return second ? gated_kernel<kAct, kBackward, true, true, true> : gated_kernel<kAct, kBackward, true, true, false>;
  if (row) return gated_kernel<kAct, kBackward, true, false, false>;
  return second ? gated_kernel<kAct, kBackward, false, true, true> : gated_kernel<kAct, kBackward, false, true, false>;
}

template <bool kBackward>
Kernel kernel_of(int act, bool row, bool col, bool second) {
  switch (act) {
    case MX_ACT_RELU: return kernel_of<MX_ACT_RELU, kBackward>(row, col, second);
    case MX_ACT_GELU: return kernel_of<MX_ACT_GELU, kBackward>(row, col, second);
    case MX_ACT_SILU: return kernel_of<MX_ACT_SILU, kBackward>(row, col, second);
    default: return kernel_of<MX_ACT_NONE, kBackward>(row, col, second);
  }
}

}  // namespace

mx_status launch_gated(const GatedLaunch& L, cudaStream_t s) {
  GatedArgs a = {};
  const bool back = L.dh != nullptr, row = L.row_data != nullptr, col = L.col_data != nullptr;
  const int64_t width = back ? 2 * L.f : L.f;
  const WaitTest test = take_wait_test();
  mx_status st = make_unit_map(&a.gate, false, L.gate_up, L.f, L.rows, L.ld, test.stages() ? kUnitRows / 2 : kUnitRows);
  if (st == MX_OK) st = make_unit_map(&a.up, false, static_cast<const uint16_t*>(L.gate_up) + L.f, L.f, L.rows, L.ld);
  if (st == MX_OK && back) st = make_unit_map(&a.dh, false, L.dh, L.f, L.rows, L.lddh);
  if (st != MX_OK) return st;
  a.q = CopyOut{static_cast<uint8_t*>(L.row_data), static_cast<uint8_t*>(L.row_scale), static_cast<uint8_t*>(L.col_data),
                static_cast<uint8_t*>(L.col_scale), width, (width + 127) / 128, L.col_pitch, (L.col_pitch + 127) / 128};
  a.rows = L.rows;
  a.f = L.f;
  const bool second = L.offsets != nullptr && col;
  const int across = units_across(back, second), per_sm = ctas_per_sm(back, second);
  a.tiles_c = (L.f + across * kUnitCols - 1) / (across * kUnitCols);
  a.tiles_r = (L.rows + kTile - 1) / kTile;
  a.offsets = L.offsets;
  a.n_groups = L.n_groups;
  a.capacity = L.col_pitch;
  a.dev_status = L.dev_status;
  a.timeout_ns = test.limit();
  const auto kern = back ? kernel_of<true>(L.act, row, col, second) : kernel_of<false>(L.act, row, col, second);
  const size_t smem = 1024 + across * (4 * (back ? 3 : 2) * 4096 + (col ? 2 * kStagedBytes : 0));
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(gated)");
  const int64_t upper = (a.tiles_r + (L.offsets ? L.n_groups : 0)) * a.tiles_c;
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(upper, static_cast<int64_t>(per_sm) * sm_count())));
  return cuda_status(launch_kernel(kern, grid, 128 * across, smem, s, 1, a),
                     back ? "mx_gated_backward_quantize launch" : "mx_gated_quantize launch");
}

}  // namespace mx
