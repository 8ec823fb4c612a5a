// mx_epilogue.cu - the backward pass of the GEMM epilogue (mx_gemm_epilogue):
//
//   dz = dy * act'(z)         (BF16, the dY that dgrad and wgrad quantise)
//   dbias = sum over rows of dy * act'(z), before dz's rounding
//
// and the epilogue alone for products over an empty contraction.
//
// Bound by HBM: dy and z read, dz written. A thread takes V neighbouring columns
// (16 bytes) and walks down the rows, so the bias's gradient stays in its
// registers and each column's terms are added in one order: the CTA's eight
// row lanes in shared memory, then one partial row per CTA in the workspace,
// added by a second launch (same inputs, same bits; no atomics).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mx_act.cuh"
#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kRowLanes = 8;      // a CTA is 32 column lanes x 8 row lanes
constexpr int kTargetCtas = 1216; // eight per SM of GB300; a constant, so the workspace's size needs no device

// V neighbouring BF16 elements (8 as one 16-byte access, or 1) as FP32 pairs.
template <int V>
struct Piece;
template <>
struct Piece<8> {
  uint4 w;
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t v = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  __device__ __forceinline__ void set(int i, float2 v) {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    (i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w) = *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ void put(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
};
template <>
struct Piece<1> {
  __nv_bfloat16 e;
  __device__ __forceinline__ float2 pair(int) const { return make_float2(__bfloat162float(e), 0.0f); }
  __device__ __forceinline__ void set(int, float2 v) { e = __float2bfloat16_rn(v.x); }
  __device__ __forceinline__ void put(__nv_bfloat16* p) const { *p = e; }
};
template <int V>
__device__ __forceinline__ Piece<V> piece_at(const __nv_bfloat16* p) {
  Piece<V> r;
  if constexpr (V == 8) r.w = *reinterpret_cast<const uint4*>(p);
  else r.e = *p;
  return r;
}

struct EpiBackwardArgs {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* z;
  __nv_bfloat16* dz;  // may be null
  float* partial;     // [gridDim.y][cols], or dbias itself when gridDim.y is 1; null: not wanted
  int64_t lddy, ldz, lddz, rows;
  int64_t cols;
};

template <int kAct, int V>
__global__ void __launch_bounds__(32 * kRowLanes) epilogue_backward_kernel(const EpiBackwardArgs a) {
  __shared__ float s[kRowLanes][32 * V + 1];
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + tx) * V;
  const int nv = static_cast<int>(min64(V, a.cols - c));
  constexpr int P = (V + 1) / 2;
  float2 sum[P];
#pragma unroll
  for (int i = 0; i < P; ++i) sum[i] = act_pair(0.0f);
  if (nv == V) {
#pragma unroll 4
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * kRowLanes + ty; row < a.rows;
         row += static_cast<int64_t>(gridDim.y) * kRowLanes) {
      const Piece<V> d = piece_at<V>(a.dy + row * a.lddy + c);
      Piece<V> z = {}, o;
      if (kAct != MX_ACT_NONE) z = piece_at<V>(a.z + row * a.ldz + c);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float2 g = d.pair(i);
        if (kAct != MX_ACT_NONE) g = __fmul2_rn(g, act_slope<kAct>(z.pair(i)));
        sum[i] = __fadd2_rn(sum[i], g);
        o.set(i, g);
      }
      if (a.dz) o.put(a.dz + row * a.lddz + c);
    }
  } else if (nv > 0) {  // the last columns of a width that is no multiple of V
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * kRowLanes + ty; row < a.rows;
         row += static_cast<int64_t>(gridDim.y) * kRowLanes) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i < nv) {
          const Piece<1> d = piece_at<1>(a.dy + row * a.lddy + c + i);
          float2 g = d.pair(0);
          if (kAct != MX_ACT_NONE) g = __fmul2_rn(g, act_slope<kAct>(piece_at<1>(a.z + row * a.ldz + c + i).pair(0)));
          (i & 1 ? sum[i / 2].y : sum[i / 2].x) += g.x;
          Piece<1> o;
          o.set(0, g);
          if (a.dz) o.put(a.dz + row * a.lddz + c + i);
        }
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int i = 0; i < V; ++i) s[ty][tx * V + i] = i & 1 ? sum[i / 2].y : sum[i / 2].x;
  __syncthreads();
  for (int j = threadIdx.x; j < 32 * V; j += 32 * kRowLanes) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 * V + j;
    if (col >= a.cols) break;
    float v = s[0][j];
#pragma unroll
    for (int y = 1; y < kRowLanes; ++y) v += s[y][j];
    a.partial[static_cast<int64_t>(blockIdx.y) * a.cols + col] = v;
  }
}

template <int kAct>
__global__ void __launch_bounds__(256) epilogue_only_kernel(const GemmEpilogue e, int64_t M, int64_t N, __nv_bfloat16* c,
                                                            int64_t ldc) {
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < M * N;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / N, col = i % N;
    float z = 0.0f;
    if (e.bias)
      z = e.bias_f32 ? static_cast<const float*>(e.bias)[col]
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(e.bias)[col]);
    if (e.preact) static_cast<__nv_bfloat16*>(e.preact)[row * e.ld_preact + col] = __float2bfloat16_rn(z);
    z = act_value<kAct>(act_pair(z)).x;
    if (e.residual) z += __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[row * e.ld_residual + col]);
    c[row * ldc + col] = __float2bfloat16_rn(z);
  }
}

// Columns of one CTA: 32 lanes of 16-byte vectors. The partial rows are counted
// for that width whatever the alignment of a call's pointers turns out to be.
int partial_rows(int64_t rows, int64_t cols) {
  const int64_t blocks = (cols + 255) / 256;
  const int64_t want = std::max<int64_t>(1, kTargetCtas / blocks);
  return static_cast<int>(std::min(want, (rows + kRowLanes - 1) / kRowLanes));
}

template <int kAct, int V>
mx_status launch_backward(const EpiBackwardArgs& a, int parts, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.cols + 32 * V - 1) / (32 * V)), static_cast<unsigned>(parts));
  cfg.blockDim = dim3(32 * kRowLanes);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_status(cudaLaunchKernelEx(&cfg, epilogue_backward_kernel<kAct, V>, a), "mx_epilogue_backward launch");
}

template <int kAct>
mx_status backward_act(const EpiBackwardArgs& a, int parts, bool vec, cudaStream_t s) {
  return vec ? launch_backward<kAct, 8>(a, parts, s) : launch_backward<kAct, 1>(a, parts, s);
}

bool vec_ok(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

}  // namespace

size_t epilogue_backward_workspace(int64_t rows, int64_t cols) {
  const int parts = partial_rows(rows, cols);
  return parts > 1 ? static_cast<size_t>(parts) * static_cast<size_t>(cols) * sizeof(float) : 0;
}

mx_status launch_epilogue_backward(const EpilogueBackwardLaunch& L, cudaStream_t s) {
  EpiBackwardArgs a;
  a.dy = static_cast<const __nv_bfloat16*>(L.dy);
  a.z = static_cast<const __nv_bfloat16*>(L.z);
  a.dz = static_cast<__nv_bfloat16*>(L.dz);
  a.lddy = L.lddy;
  a.ldz = L.ldz;
  a.lddz = L.lddz;
  a.rows = L.rows;
  a.cols = L.cols;
  const int parts = partial_rows(L.rows, L.cols);
  a.partial = !L.dbias ? nullptr : parts > 1 ? static_cast<float*>(L.ws) : L.dbias;
  const bool vec = vec_ok(L.dy, L.lddy) && (L.act == MX_ACT_NONE || vec_ok(L.z, L.ldz)) && (!L.dz || vec_ok(L.dz, L.lddz));
  mx_status st = MX_OK;
  switch (L.act) {
    case MX_ACT_RELU: st = backward_act<MX_ACT_RELU>(a, parts, vec, s); break;
    case MX_ACT_GELU: st = backward_act<MX_ACT_GELU>(a, parts, vec, s); break;
    case MX_ACT_SILU: st = backward_act<MX_ACT_SILU>(a, parts, vec, s); break;
    default: st = backward_act<MX_ACT_NONE>(a, parts, vec, s); break;
  }
  if (st != MX_OK || !L.dbias || parts == 1) return st;
  return launch_column_reduce(a.partial, parts, L.cols, 0, L.dbias, nullptr, s);
}

mx_status launch_epilogue_only(const GemmEpilogue& e, int64_t M, int64_t N, void* c, int64_t ldc, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((M * N + 255) / 256, 8 * sm_count()));
  auto kern = epilogue_only_kernel<MX_ACT_NONE>;
  if (e.act == MX_ACT_RELU) kern = epilogue_only_kernel<MX_ACT_RELU>;
  if (e.act == MX_ACT_GELU) kern = epilogue_only_kernel<MX_ACT_GELU>;
  if (e.act == MX_ACT_SILU) kern = epilogue_only_kernel<MX_ACT_SILU>;
  return cuda_status(launch_kernel(kern, grid, 256, 0, s, 1, e, M, N, static_cast<__nv_bfloat16*>(c), ldc),
                     "mx_gemm_epilogue launch (empty contraction)");
}

}  // namespace mx
