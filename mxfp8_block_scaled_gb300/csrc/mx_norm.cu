// mx_norm.cu - layer norm and root-mean-square norm over the rows of a matrix,
// forward and backward (the norm before a Linear; "DeepSeek-V3 16B FSDP2
// MXFP8/HiF8 训练设计" §1 keeps norms out of the low-precision operators).
//
//   forward   mean = sum(x) / C (0 without centring), var = sum((x - mean)^2) / C
//             rstd = 1 / sqrt(var + eps), y = (x - mean) * rstd * w + b
//   backward  h = (x - mean) * rstd, g = dy * w
//             dx = rstd * (g - sum(g) / C - h * sum(g * h) / C)  (no sum(g) without centring)
//             dw = sum over rows of dy * h, db = sum over rows of dy
//
// Everything is computed in FP32 and rounded once to the output's type. The
// variance is summed over centred values held in registers (a second sweep of
// registers, not of memory), so a mean much larger than the spread costs no
// digits.
//
// Both directions are bound by HBM (forward: x read, y written; backward: x and
// dy read, dx written); narrow rows by neither that nor the issue rate alone (below).
// By a row's number of 16-byte vectors:
//   up to 32     several rows a warp, straight into registers (no barrier at all)
//   up to 2048   a group of warps a row, fed by bulk copies through a ring of
//                stages in shared memory, the row held in the group's registers
//   above        one CTA a row, the row read again from L2 for each sweep
// BF16, measured: forward 16384 x 7168 80 us (5.9 TB/s, 88% of the copy rate),
// 16384 x 2048 27 (74%), 65536 x 128 10.5 (49%); backward 16384 x 7168 120 (88%),
// 16384 x 2048 40 (76%, 4 of it the sum of partial rows), 65536 x 128 16.7 (46%).
// FP32: 16384 x 4096 83 and 119 (97% and more). The looping kernels: 2048 x 32768
// 116 and 226 (35% and 27%).
// The backward pass keeps dw and db of its columns in registers over all rows
// of its CTA, adds its groups in shared memory and leaves one partial row per
// CTA in the workspace; a second launch adds those in a fixed order (same
// inputs, same bits; no atomics).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace {

// CTAs of the backward pass, hence partial rows of dw and db: two for each of
// GB300's 152 SMs at most (a constant, so the workspace's size needs no device).
constexpr int kMaxPartials = 304;

// Narrow rows (see below): threads of a CTA, CTAs per SM of the forward pass, and
// the sets of rows in hand, one where a lane's eight elements come one by one.
constexpr int kNarrowThreads = 256, kNarrowFwdPerSm = 3;
template <int K>
constexpr int kNarrowSets = K < 8 ? 2 : 1;

struct NormArgs {
  const void* x;
  const void* dy;      // backward
  const void* weight;  // null: 1
  const void* bias;    // null: 0
  void* out;           // y, or dx
  float* mean;         // written (forward, may be null), read (backward)
  float* rstd;
  float* partial;      // backward: [grid][2][cols], or null: no dw and db wanted
  int64_t rows;
  int64_t ldx, lddy, ldo;
  int32_t cols;
  int32_t param_f32;
  int32_t center;
  float eps;
  float inv_cols;
  int* dev_status;
  uint64_t timeout_ns;
  uint32_t withheld;  // bytes that each stage waits for in vain (the timeout's self test), else 0
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// V elements at p, of which nv exist (V or more: all); the rest read as zero.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p, int nv) {
  Pack<T, V> r;
  if (nv >= V) {
    r = *reinterpret_cast<const Pack<T, V>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i < nv) r.e[i] = p[i];
      else from_f(r.e[i], 0.0f);
    }
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& r, int nv) {
  if (nv >= V) {
    *reinterpret_cast<Pack<T, V>*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < nv) p[i] = r.e[i];
  }
}

// V parameters from column c as FP32 (dflt where there are none).
template <int V>
__device__ __forceinline__ void load_param(const void* p, bool f32, int c, int nv, float dflt, float* o) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = dflt;
  } else if (f32) {
    constexpr int W = V < 4 ? V : 4;
#pragma unroll
    for (int j = 0; j < V; j += W) {
      const Pack<float, W> v = load_pack<float, W>(static_cast<const float*>(p) + c + j, nv - j);
#pragma unroll
      for (int i = 0; i < W; ++i) o[j + i] = v.e[i];
    }
  } else {
    const Pack<__nv_bfloat16, V> v = load_pack<__nv_bfloat16, V>(static_cast<const __nv_bfloat16*>(p) + c, nv);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = to_f(v.e[i]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Keeps a row packed between two sweeps: without it the compiler carries the
// first sweep's FP32 values along, twice the registers.
template <int K, typename P>
__device__ __forceinline__ void keep_packed(P* p) {
  if constexpr (sizeof(P) >= 4) {
    uint32_t* w = reinterpret_cast<uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < static_cast<int>(K * sizeof(P) / 4); ++i) asm volatile("" : "+r"(w[i]));
  }
}

// Sums of two values over the TPR threads of a group, to all of them. `slot`:
// the group's float2 per warp, two buffers in turn (`flip`), so one barrier a
// sum is enough: nobody writes a buffer again before all have read it, which
// the barrier of the sum in between shows.
template <int TPR>
__device__ __forceinline__ void group_sum(float& a, float& b, float2* slot, int& flip, int group) {
  a = warp_sum(a);
  b = warp_sum(b);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float2* buf = slot + flip * W;
    flip ^= 1;
    const int w = (threadIdx.x % TPR) >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[w] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
    const float2 v = lane < W ? buf[lane] : make_float2(0.0f, 0.0f);
    a = warp_sum(v.x);
    b = warp_sum(v.y);
  }
}

// Rows wider than the registers of a CTA: one CTA a row, the row read three
// times (from L2 after the first). The loops count the columns that are left (nv):
// there are up to 2^31 - 1, and the place a step past the last one does not fit an
// int. All but eight BF16 at a time fit two CTAs an SM and are held to that (the
// compiler gives it up for a few registers: 63 us against 90 for 2048 x 16384 FP32).
template <int V>
constexpr int kWidePerSm = V == 8 ? 1 : 2;
template <typename T, int V>
__global__ void __launch_bounds__(1024, kWidePerSm<V>) norm_forward_wide_kernel(const NormArgs a) {
  __shared__ float2 s_sum[64];
  pdl_launch_dependents();
  pdl_wait();
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    T* out = static_cast<T*>(a.out) + row * a.ldo;
    float mean = 0.0f, sq = 0.0f, zero = 0.0f;
    if (a.center) {
      for (int nv = a.cols - threadIdx.x * V; nv > 0; nv -= 1024 * V) {
        const int c = a.cols - nv;
        const Pack<T, V> p = load_pack<T, V>(x + c, nv);
#pragma unroll
        for (int i = 0; i < V; ++i) mean += to_f(p.e[i]);
      }
      group_sum<1024>(mean, zero, s_sum, flip, 0);
      mean *= a.inv_cols;
    }
    for (int nv = a.cols - threadIdx.x * V; nv > 0; nv -= 1024 * V) {
      const int c = a.cols - nv;
      const Pack<T, V> p = load_pack<T, V>(x + c, nv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = to_f(p.e[i]) - mean;
        if (i < nv) sq = fmaf(d, d, sq);
      }
    }
    group_sum<1024>(sq, zero, s_sum, flip, 0);
    const float rstd = __frsqrt_rn(fmaf(sq, a.inv_cols, a.eps));
    for (int nv = a.cols - threadIdx.x * V; nv > 0; nv -= 1024 * V) {
      const int c = a.cols - nv;
      const Pack<T, V> p = load_pack<T, V>(x + c, nv);
      float w[V], b[V];
      load_param<V>(a.weight, a.param_f32, c, nv, 1.0f, w);
      load_param<V>(a.bias, a.param_f32, c, nv, 0.0f, b);
      Pack<T, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i) from_f(o.e[i], fmaf((to_f(p.e[i]) - mean) * rstd, w[i], b[i]));
      store_pack<T, V>(out + c, o, nv);
    }
    if (threadIdx.x == 0) {
      if (a.mean && a.center) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Wide rows: dx with one CTA a row (the row read twice) ...
template <typename T, int V>
__global__ void __launch_bounds__(1024, kWidePerSm<V>) norm_backward_wide_kernel(const NormArgs a) {
  __shared__ float2 s_sum[64];
  pdl_launch_dependents();
  pdl_wait();
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    T* out = static_cast<T*>(a.out) + row * a.ldo;
    const float mean = a.center ? a.mean[row] : 0.0f, rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int nv = a.cols - threadIdx.x * V; nv > 0; nv -= 1024 * V) {
      const int c = a.cols - nv;
      const Pack<T, V> px = load_pack<T, V>(x + c, nv), pd = load_pack<T, V>(dy + c, nv);
      float w[V];
      load_param<V>(a.weight, a.param_f32, c, nv, 1.0f, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float g = to_f(pd.e[i]) * w[i];
        s1 += g;
        s2 = fmaf(g, (to_f(px.e[i]) - mean) * rstd, s2);
      }
    }
    group_sum<1024>(s1, s2, s_sum, flip, 0);
    s1 = a.center ? s1 * a.inv_cols : 0.0f;
    s2 *= a.inv_cols;
    for (int nv = a.cols - threadIdx.x * V; nv > 0; nv -= 1024 * V) {
      const int c = a.cols - nv;
      const Pack<T, V> px = load_pack<T, V>(x + c, nv), pd = load_pack<T, V>(dy + c, nv);
      float w[V];
      load_param<V>(a.weight, a.param_f32, c, nv, 1.0f, w);
      Pack<T, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i)
        from_f(o.e[i], rstd * (to_f(pd.e[i]) * w[i] - s1 - (to_f(px.e[i]) - mean) * rstd * s2));
      store_pack<T, V>(out + c, o, nv);
    }
  }
}

// ... and dw, db by columns: CTA (bx, by) adds rows by, by + gridDim.y, ... of
// 256 * V columns.
template <typename T, int V>
__global__ void __launch_bounds__(256) norm_backward_columns_kernel(const NormArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t cols = a.cols, c = (blockIdx.x * 256 + threadIdx.x) * V;
  if (c >= cols) return;
  const int nv = cols - c;
  float dw[V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.0f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const Pack<T, V> px = load_pack<T, V>(static_cast<const T*>(a.x) + row * a.ldx + c, nv);
    const Pack<T, V> pd = load_pack<T, V>(static_cast<const T*>(a.dy) + row * a.lddy + c, nv);
    const float mean = a.center ? a.mean[row] : 0.0f, rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dw[i] = fmaf(to_f(pd.e[i]), (to_f(px.e[i]) - mean) * rstd, dw[i]);
      db[i] += to_f(pd.e[i]);
    }
  }
  float* const to_dw = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * a.cols + c;
  float* const to_db = to_dw + a.cols;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < nv) {
      to_dw[i] = dw[i];
      to_db[i] = db[i];
    }
}

// Sixteen bytes of a row as 32-bit words, and two neighbouring elements of them
// as FP32 for the packed FP32 instructions (two results an issue slot: these
// kernels are near the issue rate).
struct alignas(16) Words {
  uint32_t w[4];
};
template <typename T>
__device__ __forceinline__ float2 two_of(const Words& p, int j) {
  if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(p.w[2 * j]), __uint_as_float(p.w[2 * j + 1]));
  return make_float2(__uint_as_float(p.w[j] << 16), __uint_as_float(p.w[j] & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ void set_two(Words& p, int j, float2 v) {
  if constexpr (sizeof(T) == 4) {
    p.w[2 * j] = __float_as_uint(v.x);
    p.w[2 * j + 1] = __float_as_uint(v.y);
  } else {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    p.w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ Words words_at(const void* p) { return *reinterpret_cast<const Words*>(p); }

// ---------------------------------------------------------------------------
// Narrow rows, at most 32 vectors: TPR lanes a row, 32 / TPR rows a warp at once,
// U such sets of rows in hand and the next U on their way. A lane's columns are
// the same in every row, so it keeps their weights, and in the backward pass
// their gradients, in registers. V > 1: 16-byte vectors, one a lane (K = 1).
// V = 1: any alignment, lane r has columns r, r + TPR, ... A lane's elements are
// taken by twos. Per row the instructions are many until it has some sixteen vectors,
// hence as few lanes per row as hold it. What is left is latency: 10^6 rows of 128
// BF16 columns have 59% of the issue slots and 48% of DRAM's rate taken forward, 56%
// of both backward, with the 35% and 24% of the warps that 79 and 127 registers leave
// (the rows on their way hold half of them). With a whole warp a row, 65536 rows of 64 BF16 columns took 23 us forward and 46 backward, now 5.9 and
// 14; of 128 columns 24 and 47, now 10.5 and 16.7; 10^6 rows of 128 FP32 columns
// 161 and 242 us, 6.4 TB/s both.
// ---------------------------------------------------------------------------

template <int TPR>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Elements of a row as a lane holds them: packed while they wait, FP32 in twos.
template <typename T, int V, int TPR, int K>
struct Lane {
  static constexpr int E = V * K, P = (E + 1) / 2;
  static_assert(V == 1 || K == 1, "vectors: one a lane");
  int r, cols;
  __device__ __forceinline__ int column(int i) const { return V > 1 ? r * V + i : i * TPR + r; }
  __device__ __forceinline__ bool has(int i) const { return column(i) < cols; }  // V > 1: all of them or none
  __device__ __forceinline__ void load(Pack<T, V> (&to)[K], const T* row, bool there) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (there && has(k)) {
        to[k] = *reinterpret_cast<const Pack<T, V>*>(row + column(V > 1 ? 0 : k));
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) from_f(to[k].e[i], 0.0f);
      }
    }
  }
  __device__ __forceinline__ float2 pair(const Pack<T, V> (&p)[K], int i) const {
    if constexpr (V > 1) return make_float2(to_f(p[0].e[2 * i]), to_f(p[0].e[2 * i + 1]));
    else if constexpr (K == 1) return make_float2(to_f(p[0].e[0]), 0.0f);
    else return make_float2(to_f(p[2 * i].e[0]), to_f(p[2 * i + 1].e[0]));
  }
  __device__ __forceinline__ void store(T* row, const float2 (&v)[P]) const {
    if constexpr (V > 1) {
      if (!has(0)) return;
      Words o;
#pragma unroll
      for (int i = 0; i < P; ++i) set_two<T>(o, i, v[i]);
      *reinterpret_cast<Words*>(row + column(0)) = o;
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (has(k)) from_f(row[column(k)], k & 1 ? v[k / 2].y : v[k / 2].x);
    }
  }
  // Parameters of the lane's columns: dflt where there are none, zero past the last column.
  __device__ __forceinline__ void param(const void* p, bool f32, float dflt, float2 (&o)[P]) const {
    float f[2 * P];
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) {
      f[i] = 0.0f;
      if (i < E && has(V > 1 ? 0 : i)) {
        const int c = column(i);
        f[i] = !p ? dflt : f32 ? static_cast<const float*>(p)[c] : to_f(static_cast<const __nv_bfloat16*>(p)[c]);
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = make_float2(f[2 * i], f[2 * i + 1]);
  }
};

template <typename T, int V, int TPR, int K>
__global__ void __launch_bounds__(kNarrowThreads, kNarrowFwdPerSm) norm_forward_narrow_kernel(const NormArgs a) {
  using L = Lane<T, V, TPR, K>;
  constexpr int U = kNarrowSets<K>, P = L::P, kRows = U * 32 / TPR;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / TPR;
  const L me = {lane % TPR, a.cols};
  float2 w[P], b[P];
  me.param(a.weight, a.param_f32, 1.0f, w);
  me.param(a.bias, a.param_f32, 0.0f, b);
  const T* const x = static_cast<const T*>(a.x);
  T* const out = static_cast<T*>(a.out);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kNarrowThreads / 32) * kRows;
  int64_t base = (static_cast<int64_t>(blockIdx.x) * (kNarrowThreads / 32) + warp) * kRows;
  Pack<T, V> nxt[U][K];
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = at + u * (32 / TPR) + sub;
      me.load(nxt[u], x + row * a.ldx, row < a.rows);
    }
  };
  fetch(base);
  for (; base < a.rows; base += step) {
    Pack<T, V> cur[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < K; ++k) cur[u][k] = nxt[u][k];
    fetch(base + step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float mean = 0.0f;
      if (a.center) {
        float2 t = both(0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) t = __fadd2_rn(t, me.pair(cur[u], i));
        mean = lanes_sum<TPR>(t.x + t.y) * a.inv_cols;
      }
      float2 d[P], q = both(0.0f);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        d[i] = __fadd2_rn(me.pair(cur[u], i), both(-mean));
        if (V == 1 && !me.has(2 * i)) d[i].x = 0.0f;
        if (V == 1 && (2 * i + 1 >= K || !me.has(2 * i + 1))) d[i].y = 0.0f;
        q = __ffma2_rn(d[i], d[i], q);
      }
      const float sq = lanes_sum<TPR>(V > 1 && !me.has(0) ? 0.0f : q.x + q.y);
      const float rstd = __frsqrt_rn(fmaf(sq, a.inv_cols, a.eps));
      const int64_t row = base + u * (32 / TPR) + sub;
      if (row < a.rows) {
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = __ffma2_rn(__fmul2_rn(d[i], both(rstd)), w[i], b[i]);
        me.store(out + row * a.ldo, d);
        if (me.r == 0) {
          if (a.mean && a.center) a.mean[row] = mean;
          if (a.rstd) a.rstd[row] = rstd;
        }
      }
    }
  }
}

template <typename T, int V, int TPR, int K>
__global__ void __launch_bounds__(kNarrowThreads, 2) norm_backward_narrow_kernel(const NormArgs a) {
  using L = Lane<T, V, TPR, K>;
  constexpr int U = kNarrowSets<K>, P = L::P, kRows = U * 32 / TPR, kWarps = kNarrowThreads / 32;
  __shared__ float s_acc[2][kWarps][TPR * L::E];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / TPR;
  const L me = {lane % TPR, a.cols};
  float2 w[P], dw[P], db[P];
  me.param(a.weight, a.param_f32, 1.0f, w);
#pragma unroll
  for (int i = 0; i < P; ++i) dw[i] = db[i] = both(0.0f);
  const T* const x = static_cast<const T*>(a.x);
  const T* const dy = static_cast<const T*>(a.dy);
  T* const out = static_cast<T*>(a.out);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kRows;
  int64_t base = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRows;
  Pack<T, V> nx[U][K], nd[U][K];
  float n_mean[U], n_rstd[U];
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = at + u * (32 / TPR) + sub;
      const bool in = row < a.rows;
      me.load(nx[u], x + row * a.ldx, in);
      me.load(nd[u], dy + row * a.lddy, in);
      n_mean[u] = in && a.center ? a.mean[row] : 0.0f;
      n_rstd[u] = in ? a.rstd[row] : 0.0f;
    }
  };
  fetch(base);
  for (; base < a.rows; base += step) {
    Pack<T, V> cx[U][K], cd[U][K];
    float mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        cx[u][k] = nx[u][k];
        cd[u][k] = nd[u][k];
      }
      mean[u] = n_mean[u];
      rstd[u] = n_rstd[u];
    }
    fetch(base + step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 h[P], g[P], t1 = both(0.0f), t2 = both(0.0f);
#pragma unroll
      for (int i = 0; i < P; ++i) {  // absent elements have dy = 0 and w = 0
        const float2 d = me.pair(cd[u], i);
        h[i] = __fmul2_rn(__fadd2_rn(me.pair(cx[u], i), both(-mean[u])), both(rstd[u]));
        if (V == 1 && !me.has(2 * i)) h[i].x = 0.0f;
        if (V == 1 && (2 * i + 1 >= K || !me.has(2 * i + 1))) h[i].y = 0.0f;
        if (V > 1 && !me.has(0)) h[i] = both(0.0f);
        g[i] = __fmul2_rn(d, w[i]);
        t1 = __fadd2_rn(t1, g[i]);
        t2 = __ffma2_rn(g[i], h[i], t2);
        dw[i] = __ffma2_rn(d, h[i], dw[i]);
        db[i] = __fadd2_rn(db[i], d);
      }
      const float s1 = a.center ? lanes_sum<TPR>(t1.x + t1.y) * a.inv_cols : 0.0f;
      const float s2 = lanes_sum<TPR>(t2.x + t2.y) * a.inv_cols;
      const int64_t row = base + u * (32 / TPR) + sub;
      if (row < a.rows) {
#pragma unroll
        for (int i = 0; i < P; ++i)
          g[i] = __fmul2_rn(__ffma2_rn(h[i], both(-s2), __fadd2_rn(g[i], both(-s1))), both(rstd[u]));
        me.store(out + row * a.ldo, g);
      }
    }
  }
  if (!a.partial) return;
  // Over the warp's rows, then over the warps in order.
#pragma unroll
  for (int i = 0; i < L::E; ++i) {
    float vw = i & 1 ? dw[i / 2].y : dw[i / 2].x, vb = i & 1 ? db[i / 2].y : db[i / 2].x;
#pragma unroll
    for (int o = TPR; o < 32; o <<= 1) {
      vw += __shfl_xor_sync(0xFFFFFFFFu, vw, o);
      vb += __shfl_xor_sync(0xFFFFFFFFu, vb, o);
    }
    if (sub == 0) {
      s_acc[0][warp][me.column(i)] = vw;
      s_acc[1][warp][me.column(i)] = vb;
    }
  }
  __syncthreads();
  float* p = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  for (int i = threadIdx.x; i < 2 * a.cols; i += kNarrowThreads) {
    const int which = i >= a.cols, c = i - which * a.cols;
    float v = s_acc[which][0][c];
#pragma unroll
    for (int q = 1; q < kWarps; ++q) v += s_acc[which][q][c];
    p[i] = v;
  }
}

// ---------------------------------------------------------------------------
// Rows through shared memory: bulk copies fill a ring of stages per group while
// the group works on registers, so the bytes in flight cost no registers. A
// group is W warps; its first thread issues the copies.
//
// kElem = false: every row is a whole number of 16-byte vectors on 16-byte
// boundaries; a thread has vectors of V neighbouring elements, 32 W apart.
// kElem = true: any alignment. A bulk copy moves whole aligned 16-byte units, so
// a row's copy begins up to 15 bytes before the row and ends up to 15 after it,
// which inside the matrix are bytes of the rows next to it (or of the gap between
// them); where they would lie outside, before the first row or after the last
// one, the group reads the row itself, element by element. A thread has every
// 32 W-th element: neighbouring lanes, neighbouring elements, whatever the row's
// start in shared memory.
// ---------------------------------------------------------------------------

// Waits for a stage; a wait that runs out records MX_ERR_TIMEOUT and lets the
// CTA run on without further waits and copies. A thread whose stage has not come
// fills all of it with NaN (every bit one): what it then reads is that, or the real
// rows if they land after all, so what comes out is NaN or right, also where the
// stage passes for complete a turn of the ring later, by its parity. (The
// fill's code costs BF16 rows off the 16-byte boundaries 3-4% forward, 16384 x 2047
// 41.9 us against 40.4, the others nothing; a flag that each stage reads, 5-6%.)
__device__ __forceinline__ void stage_wait(uint64_t* bar, uint32_t parity, const NormArgs& a, volatile int32_t* gave_up,
                                           uint8_t* stages, int s, uint32_t bytes) {
  if (mbar_try_wait(bar, parity)) return;
  if (!*gave_up) {
    if (mbar_wait(bar, parity, a.timeout_ns)) return;
    *gave_up = 1;
    if (a.dev_status) atomicExch(a.dev_status, static_cast<int>(MX_ERR_TIMEOUT));
  }
#pragma unroll 1
  for (uint32_t i = 0; i < bytes; i += 16) st_shared_v4(stages + s * bytes + i, make_uint4(~0u, ~0u, ~0u, ~0u));
}

// The copies that a group's first thread has issued: one phase of full[s] each.
// After a wait that ran out it issues no more, and leave() lets the ones in
// flight land (again with a limit) before the CTA's shared memory goes away.
struct StageLog {
  uint32_t used = 0, next = 0;  // per stage: ever issued; parity of the next issue
  __device__ __forceinline__ void note(int s) {
    used |= 1u << s;
    next ^= 1u << s;
  }
  __device__ __forceinline__ void leave(uint64_t* full, int stages, const NormArgs& a, volatile int32_t* gave_up) const {
    if (!*gave_up) return;
    for (int s = 0; s < stages; ++s)
      if (used >> s & 1u) mbar_wait(&full[s], (next >> s & 1u) ^ 1u, a.timeout_ns);
  }
};

// Sums of N values over the W warps of a group, each to all of its threads.
// The first log2(N) shuffle steps halve the values a lane carries (one half of
// them goes to the lanes on either side), so N sums cost N - 1 + log2(32 / N)
// shuffles instead of 5 N. `slot`: N * W floats of the group, two buffers in
// turn, as in group_sum.
template <int N, int W>
__device__ __forceinline__ void group_totals(float (&v)[N], float* slot, int& flip, int group) {
  constexpr int L = 32 / N;  // lanes that end up with one value
  const int lane = threadIdx.x & 31;
  float t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = v[i];
#pragma unroll
  for (int n = N / 2, o = 16; n > 0; n /= 2, o /= 2) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float got = __shfl_xor_sync(0xFFFFFFFFu, upper ? t[i] : t[i + n], o);
      t[i] = (upper ? t[i + n] : t[i]) + got;
    }
  }
#pragma unroll
  for (int o = L / 2; o > 0; o /= 2) t[0] += __shfl_xor_sync(0xFFFFFFFFu, t[0], o);
  if constexpr (W > 1) {
    float* buf = slot + flip * N * W + (lane / L) * W;  // W warps' sums of this lane's value
    flip ^= 1;
    if (lane % L == 0) buf[(threadIdx.x >> 5) % W] = t[0];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * W) : "memory");
    t[0] = 0.0f;
#pragma unroll
    for (int e = 0; e < W; e += L)
      if (W >= L || lane % L < W) t[0] += buf[e + lane % L];
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) t[0] += __shfl_xor_sync(0xFFFFFFFFu, t[0], o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, t[0], i * L);
}

// A thread's place in a row: element i of its vector k.
template <typename T, int W, bool kElem>
__device__ __forceinline__ int column_of(int r, int k, int i) {
  constexpr int V = 16 / sizeof(T);
  return kElem ? (k * V + i) * 32 * W + r : (k * 32 * W + r) * V + i;
}

// Vector k of the row that begins at `row` in shared memory; what lies past the
// last column reads as zero.
template <typename T, int W, bool kElem>
__device__ __forceinline__ Words load_words(const uint8_t* row, int r, int k, int cols) {
  Words v{{0u, 0u, 0u, 0u}};
  if constexpr (!kElem) {
    if (column_of<T, W, false>(r, k, 0) < cols) v = words_at(row + (k * 32 * W + r) * 16);
  } else {
    constexpr int V = 16 / sizeof(T);
    uint32_t e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = column_of<T, W, true>(r, k, i);
      if constexpr (sizeof(T) == 4) e[i] = c < cols ? *reinterpret_cast<const uint32_t*>(row + 4 * c) : 0u;
      else e[i] = c < cols ? *reinterpret_cast<const uint16_t*>(row + 2 * c) : 0u;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) v.w[j] = e[j];
      else v.w[j] = e[2 * j] | e[2 * j + 1] << 16;
    }
  }
  return v;
}

template <typename T, int W, bool kElem>
__device__ __forceinline__ void store_words(T* row, const Words& v, int r, int k, int cols) {
  if constexpr (!kElem) {
    if (column_of<T, W, false>(r, k, 0) < cols) *reinterpret_cast<Words*>(row + column_of<T, W, false>(r, k, 0)) = v;
  } else {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = column_of<T, W, true>(r, k, i);
      if (c < cols) {
        if constexpr (sizeof(T) == 4) row[c] = __uint_as_float(v.w[i]);
        else row[c] = __ushort_as_bfloat16(static_cast<unsigned short>(v.w[i / 2] >> (16 * (i & 1))));
      }
    }
  }
}

// Parameters of elements j .. j + 3 of vector k (zero past the last column).
// kF32: they are there, in FP32.
template <typename T, int W, bool kElem, bool kF32>
__device__ __forceinline__ float4 param4(const void* p, bool f32, float dflt, int r, int k, int j, int cols) {
  float v[4];
  if constexpr (!kElem) {
    const int c = column_of<T, W, false>(r, k, j);
    if constexpr (kF32) return c < cols ? *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c)
                                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    load_param<4>(p, f32, c, cols - c, dflt, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = column_of<T, W, true>(r, k, j + i);
      if constexpr (kF32) v[i] = c < cols ? static_cast<const float*>(p)[c] : 0.0f;
      else load_param<1>(p, f32, c, cols - c, dflt, &v[i]);
    }
  }
  return make_float4(v[0], v[1], v[2], v[3]);
}

// The rows of one matrix as stages hold them.
template <typename T, bool kElem>
struct RowSource {
  const T* base;
  int64_t ld, rows;
  uint32_t bytes;  // of a row
  __device__ __forceinline__ const T* at(int64_t row) const { return base + row * ld; }
  __device__ __forceinline__ uint32_t lead(int64_t row) const {  // bytes before the row in its slot
    return kElem ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at(row)) & 15) : 0u;
  }
  static __device__ __forceinline__ uint32_t slot(uint32_t bytes) { return kElem ? ((bytes + 15) & ~15u) + 16 : bytes; }
  // Whether the copy of the row would leave the matrix.
  __device__ __forceinline__ bool edge(int64_t row) const {
    if constexpr (!kElem) return false;
    const uint32_t l = lead(row);
    return (row == 0 && l != 0) || (row == rows - 1 && ((l + bytes) & 15) != 0);
  }
  __device__ __forceinline__ uint32_t copy_bytes(int64_t row) const {
    return !kElem ? bytes : edge(row) ? 0u : (lead(row) + bytes + 15) & ~15u;
  }
  __device__ __forceinline__ void copy(uint8_t* to, int64_t row, uint64_t* bar) const {
    const uint32_t n = copy_bytes(row);
    if (n) bulk_load(to, reinterpret_cast<const uint8_t*>(at(row)) - lead(row), n, bar);
  }
  // The whole group, for an edge row.
  __device__ __forceinline__ void read(uint8_t* to, int64_t row, int r, int threads) const {
    T* const s = reinterpret_cast<T*>(to + lead(row));
    const T* const g = at(row);
    for (uint32_t c = r; c < bytes / sizeof(T); c += threads) s[c] = g[c];
  }
};

// After read(): its elements are there for the group, and for the copies that
// will overwrite them.
template <int W>
__device__ __forceinline__ void group_filled(int group) {
  fence_proxy_async_smem();
  if constexpr (W > 1) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * W) : "memory");
  else __syncwarp();
}

// Forward, two rows at a time: they share each read of weight and bias (which
// come from L1, whose bandwidth they would otherwise fill) and each barrier. A
// thread holds up to K vectors of each row.
constexpr int kFwdStages = 2;
template <int W>
constexpr int kFwdBlock = W <= 8 ? 256 : 32 * W;
// CTAs an SM: by the registers of a thread (BF16 elements one by one take more).
// Five with K = 2 spilled and took 24% longer at 16384 x 2048 BF16.
template <typename T, int W, int K, bool kElem>
constexpr int kFwdPerSm = W > 8 ? 1 : kElem && sizeof(T) == 2 ? (K == 2 ? 3 : 2) : K == 2 ? 4 : 3;

// kF32: weight and bias are both there, in FP32 (the usual case: read with no
// further questions; asking per vector cost as many instructions as the row's
// arithmetic).
template <typename T, int W, int K, bool kElem, bool kF32>
__global__ void __launch_bounds__(kFwdBlock<W>, kFwdPerSm<T, W, K, kElem>) norm_forward_ring_kernel(const NormArgs a) {
  constexpr int V = 16 / sizeof(T), G = kFwdBlock<W> / (32 * W), S = kFwdStages;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[G][S];
  __shared__ float s_sum[G][2 * 2 * W];
  __shared__ int32_t gave_up;
  pdl_launch_dependents();
  const int group = threadIdx.x / (32 * W), r = threadIdx.x % (32 * W);
  const RowSource<T, kElem> x{static_cast<const T*>(a.x), a.ldx, a.rows, static_cast<uint32_t>(a.cols) * static_cast<uint32_t>(sizeof(T))};
  const uint32_t slot = x.slot(x.bytes);
  uint8_t* const stages = ring + static_cast<size_t>(group) * S * 2 * slot;
  const int64_t pairs = (a.rows + 1) / 2, step = static_cast<int64_t>(gridDim.x) * G;
  if (r == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[group][s], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) gave_up = 0;
  __syncthreads();
  pdl_wait();
  StageLog log;
  auto issue = [&](int s, int64_t pair) {
    if (*const_cast<volatile int32_t*>(&gave_up)) return;
    log.note(s);
    const bool two = 2 * pair + 1 < a.rows;
    uint8_t* to = stages + static_cast<uint32_t>(s) * 2 * slot;
    mbar_arrive_expect_tx(&full[group][s], x.copy_bytes(2 * pair) + (two ? x.copy_bytes(2 * pair + 1) : 0u) + a.withheld);
    x.copy(to, 2 * pair, &full[group][s]);
    if (two) x.copy(to + slot, 2 * pair + 1, &full[group][s]);
  };
  int64_t pair = static_cast<int64_t>(blockIdx.x) * G + group;
  if (r == 0)
    for (int s = 0; s < S; ++s)
      if (pair + s * step < pairs) issue(s, pair + s * step);
  int s = 0, flip = 0;
  uint32_t parity = 0;
  for (; pair < pairs; pair += step) {
    stage_wait(&full[group][s], parity, a, &gave_up, stages, s, 2 * slot);
    const bool two = 2 * pair + 1 < a.rows;
    uint8_t* const from = stages + static_cast<uint32_t>(s) * 2 * slot;
    if (kElem && (x.edge(2 * pair) || (two && x.edge(2 * pair + 1)))) {
      if (x.edge(2 * pair)) x.read(from, 2 * pair, r, 32 * W);
      if (two && x.edge(2 * pair + 1)) x.read(from + slot, 2 * pair + 1, r, 32 * W);
      group_filled<W>(group);
    }
    const uint8_t* const row0 = from + x.lead(2 * pair);
    const uint8_t* const row1 = from + slot + x.lead(2 * pair + 1);
    Words p[2][K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      p[0][k] = load_words<T, W, kElem>(row0, r, k, a.cols);
      p[1][k] = load_words<T, W, kElem>(row1, r, k, two ? a.cols : 0);
    }
    float mean[2] = {0.0f, 0.0f}, sq[2] = {0.0f, 0.0f};
    if (a.center) {
      float2 t[2] = {both(0.0f), both(0.0f)};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V / 2; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q) t[q] = __fadd2_rn(t[q], two_of<T>(p[q][k], j));
      mean[0] = t[0].x + t[0].y;
      mean[1] = t[1].x + t[1].y;
      group_totals<2, W>(mean, s_sum[group], flip, group);
      mean[0] *= a.inv_cols;
      mean[1] *= a.inv_cols;
      keep_packed<K>(p[0]);
      keep_packed<K>(p[1]);
    }
    {
      const float2 minus[2] = {both(-mean[0]), both(-mean[1])};
      float2 t[2] = {both(0.0f), both(0.0f)};
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (kElem || column_of<T, W, kElem>(r, k, 0) < a.cols) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float2 d = __fadd2_rn(two_of<T>(p[q][k], j), minus[q]);
              if constexpr (kElem) {  // absent elements are no part of the variance
                if (column_of<T, W, kElem>(r, k, 2 * j) >= a.cols) d.x = 0.0f;
                if (column_of<T, W, kElem>(r, k, 2 * j + 1) >= a.cols) d.y = 0.0f;
              }
              t[q] = __ffma2_rn(d, d, t[q]);
            }
        }
      sq[0] = t[0].x + t[0].y;
      sq[1] = t[1].x + t[1].y;
    }
    group_totals<2, W>(sq, s_sum[group], flip, group);
    keep_packed<K>(p[0]);
    keep_packed<K>(p[1]);
    // Every thread of the group has its vectors in registers: the stage is free.
    if constexpr (W == 1) __syncwarp();  // group_totals has a barrier for W > 1 only; shuffles order no memory
    if (r == 0 && pair + S * step < pairs) issue(s, pair + S * step);
    if (++s == S) {
      s = 0;
      parity ^= 1;
    }
    const float rstd[2] = {__frsqrt_rn(fmaf(sq[0], a.inv_cols, a.eps)), __frsqrt_rn(fmaf(sq[1], a.inv_cols, a.eps))};
    T* const out = static_cast<T*>(a.out) + 2 * pair * a.ldo;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (column_of<T, W, kElem>(r, k, 0) >= a.cols) break;
      Words o[2];
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        asm volatile("" ::: "memory");  // four parameters at a time: hoisted, they would fill the registers
        const float4 w = param4<T, W, kElem, kF32>(a.weight, a.param_f32, 1.0f, r, k, j, a.cols);
        const float4 b = param4<T, W, kElem, kF32>(a.bias, a.param_f32, 0.0f, r, k, j, a.cols);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 lo = __fmul2_rn(__fadd2_rn(two_of<T>(p[q][k], j / 2), both(-mean[q])), both(rstd[q]));
          const float2 hi = __fmul2_rn(__fadd2_rn(two_of<T>(p[q][k], j / 2 + 1), both(-mean[q])), both(rstd[q]));
          set_two<T>(o[q], j / 2, __ffma2_rn(lo, make_float2(w.x, w.y), make_float2(b.x, b.y)));
          set_two<T>(o[q], j / 2 + 1, __ffma2_rn(hi, make_float2(w.z, w.w), make_float2(b.z, b.w)));
        }
      }
      store_words<T, W, kElem>(out, o[0], r, k, a.cols);
      if (two) store_words<T, W, kElem>(out + a.ldo, o[1], r, k, a.cols);
    }
    if (r < (two ? 2 : 1)) {
      if (a.mean && a.center) a.mean[2 * pair + r] = r ? mean[1] : mean[0];
      if (a.rstd) a.rstd[2 * pair + r] = r ? rstd[1] : rstd[0];
    }
  }
  if (r == 0) log.leave(full[group], S, a, &gave_up);
}

// Backward, R rows at a time: a stage is R neighbouring rows of x and of dy, S
// stages in flight. The rows share the barrier, the reductions and the loop's
// own instructions, which for one row are more than its arithmetic. The stage
// before is refilled after a stage's barrier, which every thread reaches only
// once it has done with that one.
template <int W>
constexpr int kBwdBlock = W <= 8 ? 256 : 32 * W;

template <typename T, int W, int K, int R, bool kElem>
__global__ void __launch_bounds__(kBwdBlock<W>, W <= 8 ? 2 : 1) norm_backward_ring_kernel(const NormArgs a, const int S) {
  constexpr int V = 16 / sizeof(T), P = V / 2, G = kBwdBlock<W> / (32 * W), kMaxS = 8;
  // What stays in a thread's registers besides dw and db: its weights, g of the
  // R rows, and h too where there is room. The rest is read or computed again.
  constexpr bool kHold = K <= 2 && (W <= 16 || (sizeof(T) == 4 && !kElem)), kHoldH = K == 1 && G == 1;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[G][kMaxS];
  __shared__ float s_sum[G][2 * 2 * R * W];
  __shared__ int32_t gave_up;
  pdl_launch_dependents();
  const int group = threadIdx.x / (32 * W), r = threadIdx.x % (32 * W);
  const uint32_t row_bytes = static_cast<uint32_t>(a.cols) * static_cast<uint32_t>(sizeof(T));
  const RowSource<T, kElem> x{static_cast<const T*>(a.x), a.ldx, a.rows, row_bytes};
  const RowSource<T, kElem> dy{static_cast<const T*>(a.dy), a.lddy, a.rows, row_bytes};
  const uint32_t slot = x.slot(row_bytes);
  uint8_t* const stages = ring + static_cast<size_t>(group) * S * 2 * R * slot;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G * R;
  if (r == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[group][s], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) gave_up = 0;
  __syncthreads();
  pdl_wait();
  StageLog log;
  auto issue = [&](int s, int64_t row) {
    if (*const_cast<volatile int32_t*>(&gave_up)) return;
    log.note(s);
    const int n = static_cast<int>(min64(R, a.rows - row));
    uint8_t* to = stages + static_cast<uint32_t>(s) * 2 * R * slot;
    uint32_t bytes = a.withheld;
    for (int q = 0; q < n; ++q) bytes += x.copy_bytes(row + q) + dy.copy_bytes(row + q);
    mbar_arrive_expect_tx(&full[group][s], bytes);
    for (int q = 0; q < n; ++q) {
      x.copy(to + q * slot, row + q, &full[group][s]);
      dy.copy(to + (R + q) * slot, row + q, &full[group][s]);
    }
  };
  int64_t row = (static_cast<int64_t>(blockIdx.x) * G + group) * R;
  if (r == 0)
    for (int s = 0; s < S; ++s)
      if (row + s * step < a.rows) issue(s, row + s * step);
  float2 dw[K * P], db[K * P];
#pragma unroll
  for (int i = 0; i < K * P; ++i) dw[i] = db[i] = both(0.0f);
  float2 w1[kHold ? K * P : 1];
  if constexpr (kHold) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < P; j += 2) {
        const float4 w = param4<T, W, kElem, false>(a.weight, a.param_f32, 1.0f, r, k, 2 * j, a.cols);
        w1[k * P + j] = make_float2(w.x, w.y);
        w1[k * P + j + 1] = make_float2(w.z, w.w);
      }
  }
  // The weights of pair j of vector k (read by fours where they are not held).
  auto weight2 = [&](int k, int j, float4& w) {
    if constexpr (kHold) return w1[kHold ? k * P + j : 0];
    if (j % 2 == 0) {
      asm volatile("" ::: "memory");
      w = a.weight && a.param_f32 ? param4<T, W, kElem, true>(a.weight, true, 1.0f, r, k, 2 * j, a.cols)
                                  : param4<T, W, kElem, false>(a.weight, a.param_f32, 1.0f, r, k, 2 * j, a.cols);
    }
    return j % 2 == 0 ? make_float2(w.x, w.y) : make_float2(w.z, w.w);
  };
  float mean[R], rstd[R];
  auto statistics = [&](int64_t at) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const bool in = at + q < a.rows;
      mean[q] = in && a.center ? a.mean[at + q] : 0.0f;
      rstd[q] = in ? a.rstd[at + q] : 0.0f;
    }
  };
  auto h_of = [&](const Words& px, int q, int j) {
    return __fmul2_rn(__fadd2_rn(two_of<T>(px, j), both(-mean[q])), both(rstd[q]));
  };
  int s = 0, flip = 0;
  uint32_t parity = 0;
  for (bool first = true; row < a.rows; row += step, first = false) {
    statistics(row);
    stage_wait(&full[group][s], parity, a, &gave_up, stages, s, 2 * R * slot);
    const int n = static_cast<int>(min64(R, a.rows - row));
    uint8_t* const from = stages + static_cast<uint32_t>(s) * 2 * R * slot;
    if constexpr (kElem) {
      bool filled = false;
      for (int q = 0; q < n; ++q) {
        if (x.edge(row + q)) x.read(from + q * slot, row + q, r, 32 * W), filled = true;
        if (dy.edge(row + q)) dy.read(from + (R + q) * slot, row + q, r, 32 * W), filled = true;
      }
      if (filled) group_filled<W>(group);
    }
    auto x_words = [&](int q, int k) {
      return load_words<T, W, kElem>(from + q * slot + x.lead(row + q), r, k, q < n ? a.cols : 0);
    };
    auto dy_words = [&](int q, int k) {
      return load_words<T, W, kElem>(from + (R + q) * slot + dy.lead(row + q), r, k, q < n ? a.cols : 0);
    };
    float2 g[kHold ? R * K * P : 1], h[kHoldH ? R * P : 1];  // h = (x - mean) rstd, g = dy w
    float sum[2 * R];  // of g, then of g h
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 t1 = both(0.0f), t2 = both(0.0f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const Words px = x_words(q, k), pd = dy_words(q, k);  // no such row or column: dy = 0 adds nothing
        if (kHold || column_of<T, W, kElem>(r, k, 0) < a.cols) {
          float4 w;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const float2 d = two_of<T>(pd, j), gj = __fmul2_rn(d, weight2(k, j, w)), hj = h_of(px, q, j);
            t1 = __fadd2_rn(t1, gj);
            t2 = __ffma2_rn(gj, hj, t2);
            dw[k * P + j] = __ffma2_rn(d, hj, dw[k * P + j]);
            db[k * P + j] = __fadd2_rn(db[k * P + j], d);
            if constexpr (kHold) g[(q * K + k) * P + j] = gj;
            if constexpr (kHoldH) h[q * P + j] = hj;
          }
        }
      }
      sum[q] = t1.x + t1.y;
      sum[R + q] = t2.x + t2.y;
    }
    group_totals<2 * R, W>(sum, s_sum[group], flip, group);
    if constexpr (W == 1) __syncwarp();  // its barrier is for W > 1 only; shuffles order no memory
    if (r == 0 && !first && row + (S - 1) * step < a.rows) issue(s == 0 ? S - 1 : s - 1, row + (S - 1) * step);
    T* out = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (q >= n) break;
      // dx = rstd g - rstd sum(g)/C - rstd (sum(g h)/C) h
      const float2 by_g = both(rstd[q]), add = both(a.center ? -rstd[q] * (sum[q] * a.inv_cols) : 0.0f),
                   by_h = both(-rstd[q] * (sum[R + q] * a.inv_cols));
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (column_of<T, W, kElem>(r, k, 0) >= a.cols) break;
        Words o, px, pd;
        if constexpr (!kHoldH) px = x_words(q, k);
        if constexpr (!kHold) pd = dy_words(q, k);
        float4 w;
#pragma unroll
        for (int j = 0; j < P; ++j) {
          float2 gj, hj;
          if constexpr (kHold) gj = g[(q * K + k) * P + j];
          else gj = __fmul2_rn(two_of<T>(pd, j), weight2(k, j, w));
          if constexpr (kHoldH) hj = h[q * P + j];
          else hj = h_of(px, q, j);
          set_two<T>(o, j, __ffma2_rn(by_h, hj, __ffma2_rn(by_g, gj, add)));
        }
        store_words<T, W, kElem>(out + q * a.ldo, o, r, k, a.cols);
      }
    }
    if (++s == S) {
      s = 0;
      parity ^= 1;
    }
  }
  if (r == 0) log.leave(full[group], S, a, &gave_up);
  if (!a.partial) return;
  float* p = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  if constexpr (G > 1) {
    // The CTA's groups, added in order, in the ring (no copy is in flight).
    float2* acc = reinterpret_cast<float2*>(ring);
    constexpr int N = 32 * W * K * P;
    __syncthreads();
    for (int q = 0; q < G; ++q) {
      if (group == q) {
#pragma unroll
        for (int i = 0; i < K * P; ++i) {
          float2* t = acc + i * 32 * W + r;
          if (q) {
            dw[i] = __fadd2_rn(dw[i], t[0]);
            db[i] = __fadd2_rn(db[i], t[N]);
          }
          t[0] = dw[i];
          t[N] = db[i];
        }
      }
      __syncthreads();
    }
    if (group != G - 1) return;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (kElem) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = column_of<T, W, true>(r, k, i);
        const float2 w = dw[k * P + i / 2], b = db[k * P + i / 2];
        if (c < a.cols) {
          p[c] = i & 1 ? w.y : w.x;
          p[a.cols + c] = i & 1 ? b.y : b.x;
        }
      }
    } else {
      const int c = column_of<T, W, false>(r, k, 0);
      if (c >= a.cols) break;
#pragma unroll
      for (int j = 0; j < P; j += 2) {
        const float2 w0 = dw[k * P + j], w1_ = dw[k * P + j + 1], b0 = db[k * P + j], b1 = db[k * P + j + 1];
        *reinterpret_cast<float4*>(p + c + 2 * j) = make_float4(w0.x, w0.y, w1_.x, w1_.y);
        *reinterpret_cast<float4*>(p + a.cols + c + 2 * j) = make_float4(b0.x, b0.y, b1.x, b1.y);
      }
    }
  }
}

mx_status norm_launched(cudaError_t e) { return cuda_status(e, "mx_layer_norm launch"); }

template <typename T, int V, int TPR, int K>
mx_status forward_narrow(const NormArgs& a, cudaStream_t s) {
  constexpr int kCtaRows = kNarrowThreads / TPR * kNarrowSets<K>;
  const int64_t grid = std::min<int64_t>((a.rows + kCtaRows - 1) / kCtaRows, kNarrowFwdPerSm * static_cast<int64_t>(sm_count()));
  return norm_launched(launch_kernel(norm_forward_narrow_kernel<T, V, TPR, K>, static_cast<unsigned>(grid), kNarrowThreads,
                                     0, s, 1, a));
}

template <typename T, int V>
mx_status forward_wide(const NormArgs& a, cudaStream_t s) {
  const int64_t grid = std::min<int64_t>(a.rows, 2 * static_cast<int64_t>(sm_count()));
  return norm_launched(launch_kernel(norm_forward_wide_kernel<T, V>, static_cast<unsigned>(grid), 1024, 0, s, 1, a));
}

// Bytes of a row's slot in a stage, and of the widest row's that W warps of K
// vectors a thread take.
template <typename T>
size_t slot_bytes(const NormArgs& a, bool elem) {
  const size_t row = static_cast<size_t>(a.cols) * sizeof(T);
  return elem ? (row + 15) / 16 * 16 + 16 : row;
}
constexpr size_t widest_slot(int W, int K, bool elem) { return static_cast<size_t>(W) * K * 512 + (elem ? 16 : 0); }

// Allows a kernel `smem` bytes of dynamic shared memory: the most that any of its
// launches takes, the same number every time, so that host threads cannot lower it
// between each other's calls of this and launches.
template <typename Kernel>
mx_status allow_smem(Kernel kern, size_t smem) {
  return cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)),
                     "cudaFuncSetAttribute(norm smem)");
}

template <typename T, int W, int K, bool kElem>
mx_status forward_ring(const NormArgs& a, cudaStream_t s) {
  constexpr int G = kFwdBlock<W> / (32 * W);
  const size_t smem = static_cast<size_t>(G) * kFwdStages * 2 * slot_bytes<T>(a, kElem);
  auto kern = a.weight && a.bias && a.param_f32 ? norm_forward_ring_kernel<T, W, K, kElem, true>
                                                : norm_forward_ring_kernel<T, W, K, kElem, false>;
  const mx_status st = allow_smem(kern, G * kFwdStages * 2 * widest_slot(W, K, kElem));
  if (st != MX_OK) return st;
  const int64_t grid = std::min<int64_t>(((a.rows + 1) / 2 + G - 1) / G, static_cast<int64_t>(sm_count()) * kFwdPerSm<T, W, K, kElem>);
  return norm_launched(launch_kernel(kern, static_cast<unsigned>(grid), kFwdBlock<W>, smem, s, 1, a));
}

// Lanes or warps per row by its number of 16-byte vectors (begun ones counted).
// BF16 rows of up to 512 take at most two vectors a thread, so that four CTAs fit
// an SM: 16384 x 2048 27.2 us against 30.8 with four vectors and half the warps,
// 16384 x 4096 46.3 against 53.0. FP32 rows, half the elements and no conversions,
// gain nothing: 16384 x 2048 48.6 against 45.0. Nor do rows of more vectors (with 16
// warps 5120 columns took 14% longer, 8192 9% less).
template <typename T, bool kElem>
mx_status forward_rows(const NormArgs& a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t n = (a.cols + V - 1) / V;
  if (n <= 32) {
    if constexpr (kElem) {
      if (a.cols <= 8) return forward_narrow<T, 1, 8, 1>(a, s);
      if (a.cols <= 16) return forward_narrow<T, 1, 8, 2>(a, s);
      if (a.cols <= 32) return forward_narrow<T, 1, 8, 4>(a, s);
      if (a.cols <= 64) return forward_narrow<T, 1, 8, 8>(a, s);
      if constexpr (V == 8)
        if (a.cols > 128) return forward_narrow<T, 1, 32, 8>(a, s);
      return forward_narrow<T, 1, 16, 8>(a, s);
    } else {
      if (n <= 4) return forward_narrow<T, V, 4, 1>(a, s);
      if (n <= 8) return forward_narrow<T, V, 8, 1>(a, s);
      if (n <= 16) return forward_narrow<T, V, 16, 1>(a, s);
      return forward_narrow<T, V, 32, 1>(a, s);
    }
  }
  if constexpr (V == 8) {
    if (n <= 64) return forward_ring<T, 1, 2, kElem>(a, s);
    if (n <= 128) return forward_ring<T, 2, 2, kElem>(a, s);
    if (n <= 256) return forward_ring<T, 4, 2, kElem>(a, s);
    if (n <= 512) return forward_ring<T, 8, 2, kElem>(a, s);
  } else {
    if (n <= 128) return forward_ring<T, 1, 4, kElem>(a, s);
    if (n <= 256) return forward_ring<T, 2, 4, kElem>(a, s);
    if (n <= 512) return forward_ring<T, 4, 4, kElem>(a, s);
  }
  if (n <= 1024) return forward_ring<T, 8, 4, kElem>(a, s);
  if (n <= 2048) return forward_ring<T, 16, 4, kElem>(a, s);
  return forward_wide<T, kElem ? 1 : V>(a, s);
}

// R rows a stage, as many stages as the share of shared memory holds (two CTAs
// an SM for groups of up to eight warps), four at most.
template <typename T, int W, int K, int R, bool kElem>
mx_status backward_ring(const NormArgs& a, int* parts, cudaStream_t s) {
  constexpr int G = kBwdBlock<W> / (32 * W), per_sm = W <= 8 ? 2 : 1;
  const size_t stage = static_cast<size_t>(G) * 2 * R * slot_bytes<T>(a, kElem);
  constexpr size_t kSmem = 212992 / per_sm;
  const int S = static_cast<int>(std::min<size_t>(4, kSmem / stage));
  static_assert(2 * G * 2 * R * widest_slot(W, K, true) <= kSmem, "a stage is refilled while another one is worked on");
  auto kern = norm_backward_ring_kernel<T, W, K, R, kElem>;
  const mx_status st = allow_smem(kern, kSmem);
  if (st != MX_OK) return st;
  const int64_t grid = std::min<int64_t>((a.rows + G * R - 1) / (G * R),
                                         std::min<int64_t>(kMaxPartials, static_cast<int64_t>(sm_count()) * per_sm));
  *parts = static_cast<int>(grid);
  return norm_launched(launch_kernel(kern, static_cast<unsigned>(grid), kBwdBlock<W>, S * stage, s, 1, a, S));
}

template <typename T, int V, int TPR, int K>
mx_status backward_narrow(const NormArgs& a, int* parts, cudaStream_t s) {
  constexpr int kCtaRows = kNarrowThreads / TPR * kNarrowSets<K>;
  const int64_t grid = std::min<int64_t>((a.rows + kCtaRows - 1) / kCtaRows,
                                         std::min<int64_t>(kMaxPartials, 2 * static_cast<int64_t>(sm_count())));
  *parts = static_cast<int>(grid);
  return norm_launched(launch_kernel(norm_backward_narrow_kernel<T, V, TPR, K>, static_cast<unsigned>(grid),
                                     kNarrowThreads, 0, s, 1, a));
}

template <typename T, int V>
mx_status backward_wide(const NormArgs& a, int* parts, cudaStream_t s) {
  const int64_t n = (a.cols + V - 1) / V;
  if (a.partial) {
    const int bx = static_cast<int>((n + 255) / 256);
    const int by = static_cast<int>(std::min<int64_t>(a.rows, std::max(1, std::min(kMaxPartials, 4 * sm_count() / bx))));
    *parts = by;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(bx, by);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const mx_status st = norm_launched(cudaLaunchKernelEx(&cfg, norm_backward_columns_kernel<T, V>, a));
    if (st != MX_OK) return st;
  }
  const int64_t grid = std::min<int64_t>(a.rows, 2 * static_cast<int64_t>(sm_count()));
  return norm_launched(launch_kernel(norm_backward_wide_kernel<T, V>, static_cast<unsigned>(grid), 1024, 0, s, 1, a));
}

template <typename T, bool kElem>
mx_status backward_rows(const NormArgs& a, int* parts, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t n = (a.cols + V - 1) / V;
  // 17 to 32 BF16 vectors: the ring, 28.0 us for 65536 x 256 against 30.0 by the
  // narrow kernel; of FP32 24.1 against 21.1, and of elements one by one 40 against 27.
  constexpr int kNarrow = kElem || V == 4 ? 32 : 16;
  if (n <= kNarrow) {
    if constexpr (kElem) {
      if (a.cols <= 8) return backward_narrow<T, 1, 8, 1>(a, parts, s);
      if (a.cols <= 16) return backward_narrow<T, 1, 8, 2>(a, parts, s);
      if (a.cols <= 32) return backward_narrow<T, 1, 8, 4>(a, parts, s);
      if (a.cols <= 64) return backward_narrow<T, 1, 8, 8>(a, parts, s);
      if constexpr (V == 8)
        if (a.cols > 128) return backward_narrow<T, 1, 32, 8>(a, parts, s);
      return backward_narrow<T, 1, 16, 8>(a, parts, s);
    } else {
      if (n <= 4) return backward_narrow<T, V, 4, 1>(a, parts, s);
      if (n <= 8) return backward_narrow<T, V, 8, 1>(a, parts, s);
      if (n <= 16) return backward_narrow<T, V, 16, 1>(a, parts, s);
      if constexpr (V == 4) return backward_narrow<T, V, 32, 1>(a, parts, s);
    }
  }
  if (n <= 32) return backward_ring<T, 1, 1, 4, kElem>(a, parts, s);
  if (n <= 64) return backward_ring<T, 2, 1, 4, kElem>(a, parts, s);
  if (n <= 128) return backward_ring<T, 4, 1, 4, kElem>(a, parts, s);
  // Half the rows a stage for BF16 elements one by one: the others' number spills
  // (16384 x 2047 63 us against 87, 16384 x 4001 111 against 116).
  constexpr int kLess = kElem && V == 8 ? 2 : 1;
  if (n <= 256) return backward_ring<T, 8, 1, 4 / kLess, kElem>(a, parts, s);
  if (n <= 512) return backward_ring<T, 8, 2, 2 / kLess, kElem>(a, parts, s);
  if (n <= 1024) return backward_ring<T, 16, 2, 2, kElem>(a, parts, s);
  if (n <= 2048) {
    // FP32: twice the warps have their weights and g in registers, 212 us against
    // 241 for 16384 x 7168. BF16 ones spill there: 184 against 158 for 8192 x 12288.
    if constexpr (V == 4 && !kElem) return backward_ring<T, 32, 2, 1, kElem>(a, parts, s);
    return backward_ring<T, 16, 4, 1, kElem>(a, parts, s);
  }
  return backward_wide<T, kElem ? 1 : V>(a, parts, s);
}

bool vec_ok(const void* p, int64_t ld, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * elem % 16 == 0;
}

NormArgs norm_args(const NormLaunch& L) {
  NormArgs a;
  a.x = L.x;
  a.dy = L.dy;
  a.weight = L.weight;
  a.bias = L.bias;
  a.out = L.out;
  a.mean = L.mean;
  a.rstd = L.rstd;
  a.partial = nullptr;
  a.rows = L.rows;
  a.ldx = L.ldx;
  a.lddy = L.lddy;
  a.ldo = L.ldo;
  a.cols = static_cast<int32_t>(L.cols);
  a.param_f32 = L.param_dtype == MX_F32;
  a.center = L.center;
  a.eps = L.eps;
  a.inv_cols = static_cast<float>(1.0 / static_cast<double>(L.cols));
  a.dev_status = L.dev_status;
  a.timeout_ns = L.timeout_ns ? L.timeout_ns : wait_timeout_ns();
  a.withheld = L.withheld;
  return a;
}

// 16-byte vectors where every row of every matrix is a whole number of them and
// starts, like the parameters, on a 16-byte boundary, else element by element. On
// aligned BF16 matrices the latter take 119 instead of 80 us for 16384 x 7168
// forward, 63 instead of 40 for 16384 x 2048 backward; FP32 ones 0-36% longer.
bool wide_access(const NormLaunch& L) {
  const int e = L.dtype == MX_F32 ? 4 : 2;
  return L.cols * e % 16 == 0 && vec_ok(L.x, L.ldx, e) && vec_ok(L.out, L.ldo, e) && (!L.dy || vec_ok(L.dy, L.lddy, e)) &&
         vec_ok(L.weight, 0, 4) && vec_ok(L.bias, 0, 4);
}

}  // namespace

mx_status launch_norm_forward(const NormLaunch& L, cudaStream_t s) {
  const NormArgs a = norm_args(L);
  const bool vec = wide_access(L);
  if (L.dtype == MX_F32) return vec ? forward_rows<float, false>(a, s) : forward_rows<float, true>(a, s);
  return vec ? forward_rows<__nv_bfloat16, false>(a, s) : forward_rows<__nv_bfloat16, true>(a, s);
}

mx_status launch_norm_backward(const NormLaunch& L, cudaStream_t s) {
  NormArgs a = norm_args(L);
  const bool vec = wide_access(L);
  const bool want = L.dweight || L.dbias;
  a.partial = want ? static_cast<float*>(L.ws) : nullptr;
  int parts = 0;
  mx_status st;
  if (L.dtype == MX_F32) st = vec ? backward_rows<float, false>(a, &parts, s) : backward_rows<float, true>(a, &parts, s);
  else st = vec ? backward_rows<__nv_bfloat16, false>(a, &parts, s) : backward_rows<__nv_bfloat16, true>(a, &parts, s);
  if (st != MX_OK || !want) return st;
  return launch_column_reduce(a.partial, parts, L.cols, L.cols, L.dweight, L.dbias, s);
}

size_t norm_backward_workspace(int64_t rows, int64_t cols) {
  return static_cast<size_t>(std::min<int64_t>(rows, kMaxPartials)) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

// ---------------------------------------------------------------------------
// Sum of partial rows
// ---------------------------------------------------------------------------

namespace {

// out[c] = sum over p of partial[p][c], c over the n0 + n1 columns of a partial
// row (the first n0 go to out0, the others to out1; null: not wanted). A CTA
// takes 8 * V columns; thread row y adds the partial rows y, y + 32, ... and a
// column's 32 sums are then added pairwise: a fixed order whatever the grid. hold_next:
// the next kernel's CTAs are not placed beside this one's.
template <int V>
__global__ void __launch_bounds__(256) column_reduce_kernel(const float* partial, int parts, int64_t n0, int64_t n1,
                                                            float* out0, float* out1, bool hold_next) {
  __shared__ float s[32][8 * V + 1];
  if (!hold_next) pdl_launch_dependents();
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int64_t n = n0 + n1, c = (static_cast<int64_t>(blockIdx.x) * 8 + tx) * V;
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.0f;
  pdl_wait();
  if (c < n) {
#pragma unroll 8
    for (int p = ty; p < parts; p += 32) {
      const Pack<float, V> q = *reinterpret_cast<const Pack<float, V>*>(partial + static_cast<int64_t>(p) * n + c);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += q.e[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s[ty][tx * V + i] = v[i];
  __syncthreads();
  // Warp w adds columns w, w + 8, ... of the tile, a lane for each thread row.
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = j * 8 + w;
    const float t = warp_sum(s[lane][col]);
    const int64_t oc = static_cast<int64_t>(blockIdx.x) * 8 * V + col;
    if (lane == 0 && oc < n) {
      float* out = oc < n0 ? out0 : out1;
      if (out) out[oc < n0 ? oc : oc - n0] = t;
    }
  }
}

}  // namespace

mx_status launch_column_reduce(const float* partial, int parts, int64_t n0, int64_t n1, float* out0, float* out1,
                               cudaStream_t s, bool hold_next) {
  const int64_t n = n0 + n1;
  const bool vec = n % 4 == 0 && (reinterpret_cast<uintptr_t>(partial) & 15) == 0;
  const int width = vec ? 32 : 8;
  return cuda_status(launch_kernel(vec ? column_reduce_kernel<4> : column_reduce_kernel<1>,
                                   static_cast<unsigned>((n + width - 1) / width), 256, 0, s, 1, partial, parts, n0, n1,
                                   out0, out1, hold_next),
                     "partial sums launch");
}

}  // namespace mx
