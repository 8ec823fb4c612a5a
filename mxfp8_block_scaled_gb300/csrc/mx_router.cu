// mx_router.cu - the router in front of the grouped products: softmax over the
// experts, top-k choice, gate weights, per-expert counts with the grouped
// calls' offsets, the balance loss, and the gradient of all of it ("DeepSeek-V3
// 16B FSDP2 MXFP8/HiF8 训练设计" §1.1: 64 routed experts, six a token; §13.4:
// the grouped products take group_list offsets).
//
//   p[t, e]    = softmax of token t's logits (0 for a logit of -inf)
//   chosen     = the top_k largest logits, ties to the lowest expert
//   w[t, j]    = p[t, chosen_j], divided by their sum when normalised
//   load[s, e] = coef * E / (top_k * S') * hits[s, e] / n_s^2, S' the sequences
//                with n_s > 0 valid tokens, hits[s, e] their choices of e
//   loss       = sum over s, e of load[s, e] * sum of p[t, e] over s's tokens
//              = coef * mean over sequences of sum over e of f_e P_e, f_e =
//                E hits / (top_k n_s), P_e = mean of p
//
//   backward   g[t, e] = dloss * load[s, e] + (gradient of the chosen weights)
//              dlogits = p * (g - sum over e of p g)   (the choice is constant)
//
// One read of the logits each way. A token's row lies in the registers of LPT
// lanes, EPL neighbouring experts each, so a warp works on 32 / LPT tokens at
// once and nothing but shuffles joins the lanes; top_k rounds of a group
// maximum choose the experts. Each CTA takes a run of tokens of one sequence and
// keeps its per-expert sums of p and counts in registers; they are added over
// the CTA in shared memory and over CTAs by two short launches, everything in a
// fixed order (same inputs, same bits; no atomics). Sums of p are FP32 over at
// most a few hundred terms at each level.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mx_internal.h"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kRouterWarps = 8;
constexpr int kRouterThreads = 32 * kRouterWarps;
constexpr int kTargetCtas = 1216;  // eight per SM of GB300; a constant, so the workspace's size needs no device
constexpr int kMinChunk = 32;      // tokens of a CTA at least
constexpr uint32_t kFull = 0xFFFFFFFFu;

// How the tokens are cut: `chunk` tokens a CTA, `per_seq` CTAs a sequence.
struct RouterPlan {
  int64_t seqs, per_seq, chunk, pitch;  // pitch: experts of a partial row (a multiple of 4)
  int64_t ctas() const { return seqs * per_seq; }
};

RouterPlan router_plan(int64_t tokens, int64_t per_seq_tokens, int64_t experts) {
  RouterPlan p;
  p.seqs = (tokens + per_seq_tokens - 1) / per_seq_tokens;
  const int64_t want = (tokens + kTargetCtas - 1) / kTargetCtas;
  p.chunk = std::max<int64_t>(kMinChunk, (want + kMinChunk - 1) / kMinChunk * kMinChunk);
  p.per_seq = (std::min(per_seq_tokens, tokens) + p.chunk - 1) / p.chunk;
  p.pitch = (experts + 3) / 4 * 4;
  return p;
}

struct RouterArgs {
  const void* logits;
  const uint8_t* mask;  // null: every token is valid
  int64_t ld, tokens, seq;
  int64_t chunk, per_seq, pitch;
  int32_t experts, top_k, normalize, vec;
  int32_t* indices;
  float* weights;
  float* part_p;     // [ctas][pitch]
  int32_t* part_n;   // [ctas][pitch]
  int32_t* part_v;   // [ctas] valid tokens
  // backward
  const float* load;      // [seqs][experts]
  const float* dweights;  // may be null
  const float* dloss;     // may be null
  void* dlogits;
  int64_t lddx;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

template <typename T>
struct alignas(16) Vec16 {
  T e[16 / sizeof(T)];
};

// Group operations over LPT neighbouring lanes (all lanes of the warp take part).
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_maxf(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (LPT == 32) return __reduce_max_sync(kFull, v);
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  if constexpr (LPT == 32) return __reduce_min_sync(kFull, v);
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Experts [first, first + EPL) of a row; those past the last read as -inf.
template <typename T, int EPL>
__device__ __forceinline__ void load_row(const T* row, int first, int experts, bool vec, float* x) {
  constexpr int W = 16 / sizeof(T);
  static_assert(EPL % W == 0, "whole 16-byte vectors");
  if (vec && first + EPL <= experts) {
#pragma unroll
    for (int j = 0; j < EPL; j += W) {
      const Vec16<T> v = *reinterpret_cast<const Vec16<T>*>(row + first + j);
#pragma unroll
      for (int i = 0; i < W; ++i) x[j + i] = to_f(v.e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = first + i < experts ? to_f(row[first + i]) : -INFINITY;
  }
}

// Softmax of a token over its group, in place; false (0 everywhere) if no logit
// is above -inf. A NaN logit makes the whole row NaN.
template <int LPT, int EPL>
__device__ __forceinline__ bool group_softmax(float* x) {
  float m = -INFINITY;
  bool any = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    m = fmaxf(m, x[i]);
    any |= !(x[i] == -INFINITY);
  }
  m = group_maxf<LPT>(m);
  any = group_max<LPT>(any ? 1u : 0u) != 0;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    x[i] = __expf(x[i] - m);
    sum += x[i];
  }
  const float inv = __frcp_rn(group_sum<LPT>(sum));
#pragma unroll
  for (int i = 0; i < EPL; ++i) x[i] = any ? x[i] * inv : 0.0f;
  return any;
}

// The tokens of this CTA: [first, end) of sequence s.
struct Run {
  int64_t first, end, s;
};
__device__ __forceinline__ Run run_of(const RouterArgs& a) {
  Run r;
  r.s = blockIdx.x / a.per_seq;
  const int64_t s0 = r.s * a.seq, s1 = min64(s0 + a.seq, a.tokens);
  r.first = s0 + (blockIdx.x % a.per_seq) * a.chunk;
  r.end = min64(r.first + a.chunk, s1);
  return r;
}

template <typename T, int LPT, int EPL>
__global__ void __launch_bounds__(kRouterThreads) router_forward_kernel(const RouterArgs a) {
  constexpr int TPW = 32 / LPT;  // tokens of a warp at a time
  __shared__ float s_p[kRouterWarps][LPT * EPL];
  __shared__ int32_t s_n[kRouterWarps][LPT * EPL];
  __shared__ int32_t s_v[kRouterWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPT, sub = lane / LPT;
  const int first = l * EPL;
  const Run run = run_of(a);
  float psum[EPL];
  int32_t hits[EPL];
  int32_t valid = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    psum[i] = 0.0f;
    hits[i] = 0;
  }
  for (int64_t t0 = run.first + warp * TPW; t0 < run.end; t0 += kRouterWarps * TPW) {
    const int64_t t = t0 + sub;
    const bool in = t < run.end;
    const bool live = in && (!a.mask || a.mask[t] != 0);
    float x[EPL];
    if (live) {
      load_row<T, EPL>(static_cast<const T*>(a.logits) + t * a.ld, first, a.experts, a.vec, x);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) x[i] = -INFINITY;
    }
    // Keys in the logits' order; 0: not to be chosen (-inf, NaN, past the last).
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t b = __float_as_uint(x[i] + 0.0f);  // -0 becomes +0
      key[i] = x[i] > -INFINITY ? b ^ (static_cast<int32_t>(b) < 0 ? 0xFFFFFFFFu : 0x80000000u) : 0u;
    }
    const bool any = group_softmax<LPT, EPL>(x);
    int32_t rank[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) rank[i] = -1;
    float chosen = 0.0f;
    int32_t found = 0;
    for (int j = 0; j < a.top_k; ++j) {
      uint32_t best = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (key[i] > best) {
          best = key[i];
          at = i;
        }
      const uint32_t top = group_max<LPT>(best);
      const uint32_t who = group_min<LPT>(best == top ? static_cast<uint32_t>(first + at) : 0xFFFFFFFFu);
      if (top != 0) {
        found = j + 1;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (who == static_cast<uint32_t>(first + i)) {
            key[i] = 0;
            rank[i] = j;
            chosen += x[i];
            ++hits[i];
          }
      }
    }
    const float scale = a.normalize ? group_sum<LPT>(chosen) : 1.0f;
    if (in) {
      int32_t* idx = a.indices + t * a.top_k;
      float* w = a.weights + t * a.top_k;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (rank[i] >= 0) {
          idx[rank[i]] = first + i;
          w[rank[i]] = a.normalize ? __fdiv_rn(x[i], scale) : x[i];
        }
      for (int j = found + l; j < a.top_k; j += LPT) {
        idx[j] = -1;
        w[j] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) psum[i] += x[i];
    valid += any;
  }
  // Over the warp's subgroups, then over the warps in order.
#pragma unroll
  for (int o = LPT; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      psum[i] += __shfl_xor_sync(kFull, psum[i], o);
      hits[i] += __shfl_xor_sync(kFull, hits[i], o);
    }
    valid += __shfl_xor_sync(kFull, valid, o);
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s_p[warp][first + i] = psum[i];
      s_n[warp][first + i] = hits[i];
    }
  }
  if (lane == 0) s_v[warp] = valid;
  __syncthreads();
  for (int e = threadIdx.x; e < a.pitch; e += kRouterThreads) {
    float p = 0.0f;
    int32_t n = 0;
    if (e < a.experts) {
      p = s_p[0][e];
      n = s_n[0][e];
#pragma unroll
      for (int w = 1; w < kRouterWarps; ++w) {
        p += s_p[w][e];
        n += s_n[w][e];
      }
    }
    a.part_p[blockIdx.x * a.pitch + e] = p;
    a.part_n[blockIdx.x * a.pitch + e] = n;
  }
  if (threadIdx.x == 0) {
    int32_t v = 0;
    for (int w = 0; w < kRouterWarps; ++w) v += s_v[w];
    a.part_v[blockIdx.x] = v;
  }
}

// One CTA per sequence: adds its CTAs' partial rows. A thread takes four experts
// of every G-th partial row; the G sums are added in order.
struct RouterSums {
  const float* part_p;
  const int32_t* part_n;
  const int32_t* part_v;
  float* seq_p;     // [seqs][pitch]: sum of p, then hits * sum of p
  int32_t* seq_n;   // [seqs][pitch]
  int32_t* seq_v;   // [seqs]
  int64_t seqs, per_seq, pitch;
  int32_t experts, top_k;
  float coef;
  int64_t* counts;
  int64_t* offsets;
  float* load;
  float* loss;
};

__global__ void __launch_bounds__(1024) router_sequence_kernel(const RouterSums a) {
  __shared__ float4 s_p[1024];
  __shared__ int4 s_n[1024];
  __shared__ int32_t s_v[32];
  pdl_launch_dependents();
  pdl_wait();
  const int lanes = static_cast<int>(a.pitch / 4), G = 1024 / lanes;
  const int e4 = threadIdx.x % lanes, g = threadIdx.x / lanes;
  const int64_t row0 = blockIdx.x * a.per_seq;
  float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  int4 n = make_int4(0, 0, 0, 0);
  if (g < G) {
#pragma unroll 4
    for (int64_t c = g; c < a.per_seq; c += G) {
      const float4 q = reinterpret_cast<const float4*>(a.part_p + (row0 + c) * a.pitch)[e4];
      const int4 m = reinterpret_cast<const int4*>(a.part_n + (row0 + c) * a.pitch)[e4];
      p.x += q.x, p.y += q.y, p.z += q.z, p.w += q.w;
      n.x += m.x, n.y += m.y, n.z += m.z, n.w += m.w;
    }
    s_p[threadIdx.x] = p;
    s_n[threadIdx.x] = n;
  }
  int32_t v = 0;
  for (int64_t c = threadIdx.x; c < a.per_seq; c += 1024) v += a.part_v[row0 + c];
  v = __reduce_add_sync(kFull, v);
  if ((threadIdx.x & 31) == 0) s_v[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < lanes) {
    const int used = static_cast<int>(min64(G, a.per_seq));
    for (int k = 1; k < used; ++k) {
      const float4 q = s_p[k * lanes + threadIdx.x];
      const int4 m = s_n[k * lanes + threadIdx.x];
      p.x += q.x, p.y += q.y, p.z += q.z, p.w += q.w;
      n.x += m.x, n.y += m.y, n.z += m.z, n.w += m.w;
    }
    reinterpret_cast<float4*>(a.seq_p + blockIdx.x * a.pitch)[threadIdx.x] = p;
    reinterpret_cast<int4*>(a.seq_n + blockIdx.x * a.pitch)[threadIdx.x] = n;
  }
  if (threadIdx.x < 32) {
    v = __reduce_add_sync(kFull, s_v[threadIdx.x]);
    if (threadIdx.x == 0) a.seq_v[blockIdx.x] = v;
  }
}

// Loads of every sequence (all CTAs); counts, offsets and loss (CTA 0).
__global__ void __launch_bounds__(512) router_finish_kernel(const RouterSums a) {
  __shared__ int32_t s_live[16];
  __shared__ float s_loss[16];
  __shared__ int64_t s_scan[512];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t live = 0;
  for (int64_t s = tid; s < a.seqs; s += 512) live += a.seq_v[s] > 0;
  live = __reduce_add_sync(kFull, live);
  if (lane == 0) s_live[warp] = live;
  __syncthreads();
  live = 0;
  for (int w = 0; w < 16; ++w) live += s_live[w];
  const float factor = a.coef * (static_cast<float>(a.experts) / (static_cast<float>(a.top_k) * static_cast<float>(max(live, 1))));
  const int64_t total = a.seqs * a.experts;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 512 + tid; i < total; i += static_cast<int64_t>(gridDim.x) * 512) {
    const int64_t s = i / a.experts, e = i % a.experts;
    const float n = static_cast<float>(max(a.seq_v[s], 1));
    a.load[i] = factor * static_cast<float>(a.seq_n[s * a.pitch + e]) / (n * n);
  }
  if (blockIdx.x != 0) return;
  float loss = 0.0f;
  int64_t count = 0;
  if (tid < a.experts) {
#pragma unroll 4
    for (int64_t s = 0; s < a.seqs; ++s) {
      const float n = static_cast<float>(max(a.seq_v[s], 1));
      const int32_t hit = a.seq_n[s * a.pitch + tid];
      count += hit;
      loss += factor * static_cast<float>(hit) / (n * n) * a.seq_p[s * a.pitch + tid];
    }
    a.counts[tid] = count;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(kFull, loss, o);
  if (lane == 0) s_loss[warp] = loss;
  s_scan[tid] = count;
  __syncthreads();
  for (int o = 1; o < 512; o <<= 1) {
    const int64_t before = tid >= o ? s_scan[tid - o] : 0;
    __syncthreads();
    s_scan[tid] += before;
    __syncthreads();
  }
  if (tid < a.experts) a.offsets[tid + 1] = s_scan[tid];
  if (tid == 0) {
    a.offsets[0] = 0;
    loss = 0.0f;
    for (int w = 0; w < 16; ++w) loss += s_loss[w];
    *a.loss = loss;
  }
}

template <typename T, int LPT, int EPL>
__global__ void __launch_bounds__(kRouterThreads) router_backward_kernel(const RouterArgs a) {
  constexpr int TPW = 32 / LPT;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPT, sub = lane / LPT;
  const int first = l * EPL;
  const Run run = run_of(a);
  float load[EPL];
  const float dloss = a.dloss ? *a.dloss : 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) load[i] = first + i < a.experts ? dloss * a.load[run.s * a.experts + first + i] : 0.0f;
  for (int64_t t0 = run.first + warp * TPW; t0 < run.end; t0 += kRouterWarps * TPW) {
    const int64_t t = t0 + sub;
    const bool in = t < run.end;
    const bool live = in && (!a.mask || a.mask[t] != 0);
    float x[EPL], g[EPL];
    if (live) {
      load_row<T, EPL>(static_cast<const T*>(a.logits) + t * a.ld, first, a.experts, a.vec, x);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) x[i] = -INFINITY;
    }
    const bool any = group_softmax<LPT, EPL>(x);
#pragma unroll
    for (int i = 0; i < EPL; ++i) g[i] = load[i];
    if (a.dweights) {
      // The chosen weights' gradients at their experts. When normalised, w_j =
      // p_j / z: dp_j = (dw_j - sum_i w_i dw_i) / z, with every dw taken against
      // the first one so that equal ones (a single choice too) cancel exactly.
      float dw[EPL];
      uint32_t mine = 0;
      const int64_t at = t * a.top_k;
      const float d0 = live && a.normalize ? a.dweights[at] : 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) dw[i] = 0.0f;
      for (int j = 0; j < a.top_k; ++j) {
        const int e = live ? a.indices[at + j] - first : -1;
        const float d = live ? a.dweights[at + j] - d0 : 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (e == i) {
            dw[i] = d;
            mine |= 1u << i;
          }
      }
      if (a.normalize) {
        float z = 0.0f, s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (mine >> i & 1u) {
            z += x[i];
            s = fmaf(x[i], dw[i], s);
          }
        const float inv = __frcp_rn(group_sum<LPT>(z));
        s = group_sum<LPT>(s) * inv;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (mine >> i & 1u) g[i] = fmaf(dw[i] - s, inv, g[i]);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) g[i] += dw[i];
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) dot = fmaf(x[i], g[i], dot);
    dot = group_sum<LPT>(dot);
    if (in) {
      T* out = static_cast<T*>(a.dlogits) + t * a.lddx + first;
      constexpr int W = 16 / sizeof(T);
      if (a.vec && first + EPL <= a.experts) {
#pragma unroll
        for (int j = 0; j < EPL; j += W) {
          Vec16<T> v;
#pragma unroll
          for (int i = 0; i < W; ++i) from_f(v.e[i], any ? x[j + i] * (g[j + i] - dot) : 0.0f);
          *reinterpret_cast<Vec16<T>*>(out + j) = v;
        }
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (first + i < a.experts) from_f(out[i], any ? x[i] * (g[i] - dot) : 0.0f);
      }
    }
  }
}

template <typename T, int LPT, int EPL>
mx_status run_cfg(const RouterArgs& a, int64_t ctas, bool backward, cudaStream_t s) {
  auto kern = backward ? router_backward_kernel<T, LPT, EPL> : router_forward_kernel<T, LPT, EPL>;
  return cuda_status(launch_kernel(kern, static_cast<unsigned>(ctas), kRouterThreads, 0, s, 1, a), "mx_router launch");
}

// Lanes a token by the number of experts, eight experts a lane (sixteen above 256).
template <typename T>
mx_status run_any(const RouterArgs& a, int64_t ctas, bool backward, cudaStream_t s) {
  if (a.experts <= 32) return run_cfg<T, 4, 8>(a, ctas, backward, s);
  if (a.experts <= 64) return run_cfg<T, 8, 8>(a, ctas, backward, s);
  if (a.experts <= 128) return run_cfg<T, 16, 8>(a, ctas, backward, s);
  if (a.experts <= 256) return run_cfg<T, 32, 8>(a, ctas, backward, s);
  return run_cfg<T, 32, 16>(a, ctas, backward, s);
}

RouterArgs router_args(const RouterLaunch& L, const RouterPlan& p) {
  RouterArgs a = {};
  a.logits = L.logits;
  a.mask = L.mask;
  a.ld = L.ld;
  a.tokens = L.tokens;
  a.seq = L.tokens_per_seq;
  a.chunk = p.chunk;
  a.per_seq = p.per_seq;
  a.pitch = p.pitch;
  a.experts = L.experts;
  a.top_k = L.top_k;
  a.normalize = L.normalize;
  const int64_t bytes = L.dtype == MX_F32 ? 4 : 2;
  const auto wide = [&](const void* q, int64_t ld) {
    return !q || ((reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld * bytes % 16 == 0);
  };
  a.vec = wide(L.logits, L.ld) && wide(L.dlogits, L.lddx);
  a.indices = L.indices;
  a.weights = L.weights;
  a.load = L.load;
  a.dweights = L.dweights;
  a.dloss = L.dloss;
  a.dlogits = L.dlogits;
  a.lddx = L.lddx;
  return a;
}

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

// Partial rows of p and counts, valid tokens, then the same per sequence.
size_t router_workspace(int64_t tokens, int64_t tokens_per_seq, int experts) {
  const RouterPlan p = router_plan(tokens, tokens_per_seq, experts);
  return static_cast<size_t>((p.ctas() + p.seqs) * p.pitch * 8 + round16(p.ctas() * 4) + round16(p.seqs * 4));
}

bool router_fits(int64_t tokens, int64_t tokens_per_seq, int experts) {
  return router_plan(tokens, tokens_per_seq, experts).ctas() <= 0x7FFFFFFF;
}

mx_status launch_router_forward(const RouterLaunch& L, cudaStream_t s) {
  const RouterPlan p = router_plan(L.tokens, L.tokens_per_seq, L.experts);
  RouterArgs a = router_args(L, p);
  char* w = static_cast<char*>(L.ws);
  const auto take = [&](int64_t bytes) {
    char* at = w;
    w += bytes;
    return at;
  };
  const int64_t part = p.ctas() * p.pitch * 4, seq = p.seqs * p.pitch * 4;
  RouterSums q = {};
  q.part_p = a.part_p = reinterpret_cast<float*>(take(part));
  q.part_n = a.part_n = reinterpret_cast<int32_t*>(take(part));
  q.seq_p = reinterpret_cast<float*>(take(seq));
  q.seq_n = reinterpret_cast<int32_t*>(take(seq));
  q.part_v = a.part_v = reinterpret_cast<int32_t*>(take(round16(p.ctas() * 4)));
  q.seq_v = reinterpret_cast<int32_t*>(take(round16(p.seqs * 4)));
  q.seqs = p.seqs;
  q.per_seq = p.per_seq;
  q.pitch = p.pitch;
  q.experts = L.experts;
  q.top_k = L.top_k;
  q.coef = L.coef;
  q.counts = L.counts;
  q.offsets = L.offsets;
  q.load = L.load;
  q.loss = L.loss;
  mx_status st = L.dtype == MX_F32 ? run_any<float>(a, p.ctas(), false, s) : run_any<__nv_bfloat16>(a, p.ctas(), false, s);
  if (st != MX_OK) return st;
  st = cuda_status(launch_kernel(router_sequence_kernel, static_cast<unsigned>(p.seqs), 1024, 0, s, 1, q),
                   "mx_router launch (sequences)");
  if (st != MX_OK) return st;
  const int64_t grid = std::min<int64_t>(sm_count(), (p.seqs * L.experts + 2047) / 2048);
  return cuda_status(launch_kernel(router_finish_kernel, static_cast<unsigned>(grid), 512, 0, s, 1, q),
                     "mx_router launch (loss)");
}

mx_status launch_router_backward(const RouterLaunch& L, cudaStream_t s) {
  const RouterPlan p = router_plan(L.tokens, L.tokens_per_seq, L.experts);
  const RouterArgs a = router_args(L, p);
  return L.dtype == MX_F32 ? run_any<float>(a, p.ctas(), true, s) : run_any<__nv_bfloat16>(a, p.ctas(), true, s);
}

}  // namespace mx
