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
// once and nothing but shuffles joins the lanes. The work is bound by issued
// instructions before it is by memory, so the choice is made on one 32-bit key
// per logit that also holds the expert: the lanes sort their keys once and
// top_k rounds of a group maximum take the heads. Each CTA takes a run of tokens
// of one sequence; its sums of p stay in registers, are added over the CTA in
// shared memory and over CTAs by one or two short launches, in a fixed order (same
// inputs, same bits). Only whole numbers are added by atomics, in shared memory.
// Sums of p are FP32 over at most a few hundred terms at each level.

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
constexpr int kTargetCtas = 608;   // four per SM of GB300; a constant, so the workspace's size needs no device
constexpr int kMinChunk = 32;      // tokens of a CTA at least, and what a chunk is a multiple of
// The backward pass leaves no partial rows, so its cut is its own: five CTAs per
// SM, chunks of whole rounds of a CTA's warps (65536 tokens of 256 experts in
// chunks of 128, 512 CTAs, took 11% longer: some SMs had four of them, some three).
constexpr int kBackwardCtas = 760;
constexpr uint32_t kFull = 0xFFFFFFFFu;

// How the tokens are cut: `chunk` tokens a CTA (a multiple of step, about `target`
// CTAs in all), `per_seq` CTAs a sequence.
struct RouterPlan {
  int64_t seqs, per_seq, chunk, pitch;  // pitch: experts of a partial row (a multiple of 4)
  int64_t ctas() const { return seqs * per_seq; }
};

RouterPlan router_plan(int64_t tokens, int64_t per_seq_tokens, int64_t experts, int64_t target = kTargetCtas,
                       int64_t step = kMinChunk) {
  RouterPlan p;
  p.seqs = (tokens + per_seq_tokens - 1) / per_seq_tokens;
  const int64_t want = (tokens + target - 1) / target;
  p.chunk = std::max<int64_t>(kMinChunk, (want + step - 1) / step * step);
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

// A logit as an unsigned number of the same order; -0 counts as +0. -inf (and a
// NaN with its sign bit set) gives at most kNoKey, every number more; other
// NaNs come out above +inf.
constexpr uint32_t kNoKey = 0x007FFFFFu, kInfKey = 0xFF800000u;
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// exp(x) for x <= 0 with results below 2^-126 flushed to zero.
__device__ __forceinline__ float exp_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}

__device__ __forceinline__ void order_pair(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}

// Descending: halves sorted, then merged (the second half met in reverse, which
// leaves two bitonic halves).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t* k) {
  if constexpr (N > 1) {
    sort_keys<N / 2>(k);
    sort_keys<N / 2>(k + N / 2);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) order_pair(k[i], k[N - 1 - i]);
#pragma unroll
    for (int q = N / 4; q >= 1; q /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i & q) == 0) order_pair(k[i], k[i + q]);
  }
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

// 65536 tokens, 64 FP32 experts, six choices: 16.5 us, 68% of the issue slots, a
// third of the instructions in the six rounds of the choice; 20.5 us with the sums.
// Some of the others move spilled registers: four CTAs an SM leave 64 a thread, and
// x, ahead, key and psum are alive together. Bytes stored and loaded per thread, for
// 4, 8, 16 and 32 lanes a token: FP32 52/76, 56/80, 56/80, 12/12; BF16 52/76, 32/44,
// 32/44, 12/12.
template <typename T, int LPT, int EPL>
__global__ void __launch_bounds__(kRouterThreads, EPL == 8 ? 4 : 2) router_forward_kernel(const RouterArgs a) {
  constexpr int TPW = 32 / LPT;   // tokens of a warp at a time
  constexpr int E = LPT * EPL;    // experts that fit
  // A packed key: the logit's key without its lowest bits, which hold E - 1 -
  // expert, so that the larger key wins and ties go to the lowest expert. BF16
  // logits lose nothing by it. FP32 ones do: where two keys that meet in the
  // choice agree in all that is left of their logits, the token is done again
  // with whole keys.
  constexpr uint32_t kLow = E - 1;
  static_assert((E & (E - 1)) == 0 && E <= 512, "bits for the expert");
  constexpr bool kExact = sizeof(T) == 2;
  __shared__ float s_p[kRouterWarps][E];
  __shared__ int32_t s_n[E];
  __shared__ int32_t s_v[kRouterWarps];
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < E; e += kRouterThreads) s_n[e] = 0;
  __syncthreads();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPT, sub = lane / LPT;
  const int first = l * EPL;
  const Run run = run_of(a);
  float psum[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) psum[i] = 0.0f;
  int32_t valid = 0;
  // The next token's row is on its way while this one is worked on. Places move
  // on by fixed steps: row, choices and weights of token t0 + sub.
  constexpr int kStep = kRouterWarps * TPW;
  const int64_t t0 = run.first + warp * TPW + sub;
  const int tokens = static_cast<int>(run.end - run.first);
  const T* row = static_cast<const T*>(a.logits) + t0 * a.ld;
  const uint8_t* live_at = a.mask ? a.mask + t0 : nullptr;
  int32_t* idx = a.indices + t0 * a.top_k;
  float* w = a.weights + t0 * a.top_k;
  const int64_t row_step = kStep * a.ld;
  const int choice_step = kStep * a.top_k;
  const bool few = a.top_k <= LPT;  // a lane has one choice at most
  float ahead[EPL];
  bool live_ahead;
  auto fetch = [&](bool there, const T* from) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) ahead[i] = -INFINITY;
    live_ahead = there && (!a.mask || *live_at != 0);
    if (live_ahead) load_row<T, EPL>(from, first, a.experts, a.vec, ahead);
  };
  fetch(warp * TPW + sub < tokens, row);
  for (int q = warp * TPW; q < tokens; q += kStep, row += row_step, idx += choice_step, w += choice_step) {
    const bool in = q + sub < tokens;
    float x[EPL];  // a token left out is -inf throughout
    uint32_t key[EPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      x[i] = ahead[i];
      m = fmaxf(m, x[i]);
      key[i] = (order_key(x[i]) & ~kLow) | (kLow - static_cast<uint32_t>(first + i));
    }
    const bool live = live_ahead;
    if (a.mask) live_at += kStep;
    fetch(q + sub + kStep < tokens, row + row_step);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    sort_keys<EPL>(key);
    // Lane j % LPT holds choice j (the last such one; where there are more, each
    // is written as it is made).
    uint32_t last = 0, mine = 0, apart = kFull;
    uint32_t top = 0;
    for (int j = 0; j < a.top_k; ++j) {
      const uint32_t best = group_max<LPT>(key[0]);
      if (!kExact) apart = min(apart, best ^ last);
      last = best;
      if (j == 0) top = best;
      if (few) {
        if (j == l) mine = best;
      } else if (j % LPT == l && in) {
        idx[j] = best > kNoKey ? static_cast<int32_t>(kLow - (best & kLow)) : -1;
      }
      if (key[0] == best) {  // one lane: keys differ by their experts
#pragma unroll
        for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
        key[EPL - 1] = 0;
      }
    }
    // The first one not chosen may be as close to the last one chosen.
    if (!kExact) apart = min(apart, group_max<LPT>(key[0]) ^ last);
    bool any = top > kNoKey;
    int e0 = mine > kNoKey ? static_cast<int>(kLow - (mine & kLow)) : -1;
    // Once more with whole keys, if rounding or a NaN may have changed the
    // choice (a row of -inf alone does not count).
    const bool again = (!kExact && any && apart <= kLow) || top >= kInfKey;
    if (__any_sync(kFull, again || (live && !any))) {
      bool nan = false;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        nan |= x[i] != x[i];
        key[i] = x[i] > -INFINITY ? order_key(x[i]) : 0u;
      }
      any |= group_max<LPT>(nan ? 1u : 0u) != 0;
      for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (key[i] > best) {
            best = key[i];
            at = i;
          }
        const uint32_t most = group_max<LPT>(best);
        const uint32_t who = group_min<LPT>(best == most ? static_cast<uint32_t>(first + at) : kFull);
        if (j % LPT == l) {
          e0 = most != 0 ? static_cast<int>(who) : -1;
          if (!few && in) idx[j] = e0;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (most != 0 && who == static_cast<uint32_t>(first + i)) key[i] = 0;
      }
    }
    if (!any) m = 0.0f;  // the row's exponentials are then zero
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      x[i] = exp_of(x[i] - m);
      sum += x[i];
    }
    sum = group_sum<LPT>(sum);
    const float inv = any ? __frcp_rn(sum) : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) psum[i] = fmaf(x[i], inv, psum[i]);
    valid += any;
    // The chosen weights, p computed again from the logit.
    if (few) {
      float p = 0.0f;
      if (e0 >= 0) {
        p = exp_of(to_f(row[e0]) - m) * inv;
        atomicAdd(&s_n[e0], 1);
      }
      if (a.normalize) {
        const float all = group_sum<LPT>(p);
        if (e0 >= 0) p *= __frcp_rn(all);
      }
      if (in && l < a.top_k) {
        idx[l] = e0;
        w[l] = p;
      }
    } else {
      float all = 0.0f;
      for (int j = l; j < a.top_k; j += LPT) {
        const int e = in ? idx[j] : -1;
        if (e >= 0) {
          all += exp_of(to_f(row[e]) - m) * inv;
          atomicAdd(&s_n[e], 1);
        }
      }
      const float scale = a.normalize ? __frcp_rn(group_sum<LPT>(all)) : 1.0f;
      if (in)
        for (int j = l; j < a.top_k; j += LPT) {
          const int e = idx[j];
          w[j] = e >= 0 ? exp_of(to_f(row[e]) - m) * inv * scale : 0.0f;
        }
    }
  }
  // Over the warp's subgroups, then over the warps in order.
#pragma unroll
  for (int o = LPT; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) psum[i] += __shfl_xor_sync(kFull, psum[i], o);
    valid += __shfl_xor_sync(kFull, valid, o);
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s_p[warp][first + i] = psum[i];
  }
  if (lane == 0) s_v[warp] = valid;
  __syncthreads();
  for (int e = threadIdx.x; e < a.pitch; e += kRouterThreads) {
    float p = 0.0f;
    int32_t n = 0;
    if (e < a.experts) {
      n = s_n[e];
      p = s_p[0][e];
#pragma unroll
      for (int w = 1; w < kRouterWarps; ++w) p += s_p[w][e];
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

// The sums of a sequence over its CTAs' partial rows: a thread takes four experts
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

struct SumScratch {
  float4 p[1024];
  int4 n[1024];
  int32_t v[32];
};

// Sequence s: one CTA of 1024 threads adds the partial rows of its CTAs.
__device__ __forceinline__ void add_sequence(const RouterSums& a, int64_t s, SumScratch& sh) {
  const int lanes = static_cast<int>(a.pitch / 4), G = 1024 / lanes;
  const int e4 = threadIdx.x % lanes, g = threadIdx.x / lanes;
  const int64_t row0 = s * a.per_seq;
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
    sh.p[threadIdx.x] = p;
    sh.n[threadIdx.x] = n;
  }
  int32_t v = 0;
  for (int64_t c = threadIdx.x; c < a.per_seq; c += 1024) v += a.part_v[row0 + c];
  v = __reduce_add_sync(kFull, v);
  if ((threadIdx.x & 31) == 0) sh.v[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < lanes) {
    const int used = static_cast<int>(min64(G, a.per_seq));
    for (int k = 1; k < used; ++k) {
      const float4 q = sh.p[k * lanes + threadIdx.x];
      const int4 m = sh.n[k * lanes + threadIdx.x];
      p.x += q.x, p.y += q.y, p.z += q.z, p.w += q.w;
      n.x += m.x, n.y += m.y, n.z += m.z, n.w += m.w;
    }
    reinterpret_cast<float4*>(a.seq_p + s * a.pitch)[threadIdx.x] = p;
    reinterpret_cast<int4*>(a.seq_n + s * a.pitch)[threadIdx.x] = n;
  }
  if (threadIdx.x < 32) {
    v = __reduce_add_sync(kFull, sh.v[threadIdx.x]);
    if (threadIdx.x == 0) a.seq_v[s] = v;
  }
  __syncthreads();  // the scratch is free again
}

struct FinishScratch {
  int32_t live[32];
  float loss[32];
  int64_t count[1024];
  int64_t warp[32];
};

// Loads of every sequence (each CTA takes every gridDim-th one of G at a time);
// counts, offsets and loss (CTA 0, over all of them). A thread has one expert.
__device__ __forceinline__ void finish(const RouterSums& a, int width, FinishScratch& sh) {
  // width: a power of two at least the number of experts
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, e = tid & (width - 1), g = tid / width, G = 1024 / width;
  int32_t live = 0;
  for (int64_t s = tid; s < a.seqs; s += 1024) live += a.seq_v[s] > 0;
  live = __reduce_add_sync(kFull, live);
  if (lane == 0) sh.live[warp] = live;
  __syncthreads();
  live = __reduce_add_sync(kFull, sh.live[lane]);
  const float factor = a.coef * (static_cast<float>(a.experts) / (static_cast<float>(a.top_k) * static_cast<float>(max(live, 1))));
  float loss = 0.0f;
  int64_t count = 0;
  if (e < a.experts) {
    const bool all = blockIdx.x == 0;  // CTA 0 also needs the other CTAs' sequences
#pragma unroll 4
    for (int64_t s = all ? g : g + static_cast<int64_t>(blockIdx.x) * G; s < a.seqs; s += all ? G : static_cast<int64_t>(gridDim.x) * G) {
      const float n = static_cast<float>(max(a.seq_v[s], 1));
      const int32_t hit = a.seq_n[s * a.pitch + e];
      const float load = factor * static_cast<float>(hit) / (n * n);
      if (!all || s / G % gridDim.x == 0) a.load[s * a.experts + e] = load;
      if (all) {
        count += hit;
        loss = fmaf(load, a.seq_p[s * a.pitch + e], loss);
      }
    }
  }
  if (blockIdx.x != 0) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(kFull, loss, o);
  if (lane == 0) sh.loss[warp] = loss;
  sh.count[tid] = count;
  __syncthreads();
  if (tid == 0) {
    loss = 0.0f;
    for (int w = 0; w < 32; ++w) loss += sh.loss[w];
    *a.loss = loss;
    a.offsets[0] = 0;
  }
  // Experts' totals and their running sums: over the lanes, then over the warps.
  count = 0;
  if (tid < a.experts) {
    for (int q = 0; q < G; ++q) count += sh.count[q * width + tid];
    a.counts[tid] = count;
  }
  int64_t run = count;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t before = __shfl_up_sync(kFull, run, o);
    if (lane >= o) run += before;
  }
  if (lane == 31) sh.warp[warp] = run;
  __syncthreads();
  for (int w = 0; w < warp; ++w) run += sh.warp[w];
  if (tid < a.experts) a.offsets[tid + 1] = run;
}

__global__ void __launch_bounds__(1024) router_sequence_kernel(const RouterSums a) {
  __shared__ SumScratch sh;
  pdl_launch_dependents();
  pdl_wait();
  add_sequence(a, blockIdx.x, sh);
}

__global__ void __launch_bounds__(1024) router_finish_kernel(const RouterSums a, int width) {
  __shared__ FinishScratch sh;
  pdl_launch_dependents();
  pdl_wait();
  finish(a, width, sh);
}

// Both in one launch for few sequences: a cluster of eight CTAs adds them, meets
// at the cluster's barrier (which makes their sums visible to all of it) and
// finishes.
constexpr int kTailCtas = 8, kTailSeqs = 32;
__global__ void __launch_bounds__(1024) router_tail_kernel(const RouterSums a, int width) {
  __shared__ union {
    SumScratch sum;
    FinishScratch finish;
  } sh;
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t s = blockIdx.x; s < a.seqs; s += kTailCtas) add_sequence(a, s, sh.sum);
  cluster_sync();
  finish(a, width, sh.finish);
}

// Sums of four values over a group, to all of its lanes: two halving steps, then
// the rest of the tree on one value.
template <int LPT>
__device__ __forceinline__ void group_sum4(float (&v)[4]) {
  constexpr int L = LPT / 4;  // lanes that end up with one value
  const int l = threadIdx.x % LPT, base = (threadIdx.x & 31) - l;
  const bool up = (l & LPT / 2) != 0, up2 = (l & LPT / 4) != 0;
  float a = (up ? v[2] : v[0]) + __shfl_xor_sync(kFull, up ? v[0] : v[2], LPT / 2);
  const float b = (up ? v[3] : v[1]) + __shfl_xor_sync(kFull, up ? v[1] : v[3], LPT / 2);
  a = (up2 ? b : a) + __shfl_xor_sync(kFull, up2 ? a : b, LPT / 4);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(kFull, a, base + i * L);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The maximum over a group; NaNs are passed over.
template <int LPT>
__device__ __forceinline__ float group_max_f(float v) {
  if constexpr (LPT == 32) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  }
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

__device__ __forceinline__ void set_pair(float* d, float2 v) { *reinterpret_cast<float2*>(d) = v; }
__device__ __forceinline__ void set_pair(__nv_bfloat16* d, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(d) = __floats2bfloat162_rn(v.x, v.y);
}

// With e = exp(x - m) and p = e / sum(e), one reduction over the group gives
// sum(e), sum(e load), and over the chosen ones z = sum(e) and s = sum(e dw).
// Not normalised: dot = sum(p load) + sum(p dw). Normalised (w = e / z): the
// chosen ones' dp = (dw - s/z) / (z/sum), whose p-weighted sum is zero, so dot =
// sum(p load); every dw is taken against the first one, so that equal ones (a
// single choice too) cancel exactly. The chosen elements' results are computed
// by the lanes that hold their dw and put over the row's in shared memory.
//
// Bound by issued instructions (70% of the slots) for BF16: 65536 tokens of 256
// experts take 23 us (3.1 TB/s of the 71 MB); by memory for FP32: 27 us, 77% of
// the copy rate. Loading the next token's row ahead cost registers, hence warps,
// and 20-50% of the time.
template <typename T, int LPT, int EPL>
__global__ void __launch_bounds__(kRouterThreads, EPL == 8 ? 5 : 2) router_backward_kernel(const RouterArgs a) {
  constexpr int TPW = 32 / LPT, E = LPT * EPL, W = 16 / sizeof(T), P = EPL / 2, kStep = kRouterWarps * TPW;
  __shared__ __align__(16) T s_row[kStep][E];
  __shared__ __align__(16) float s_load[E];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPT, sub = lane / LPT;
  const int first = l * EPL;
  const Run run = run_of(a);
  const float dloss = a.dloss ? *a.dloss : 0.0f;
  for (int e = threadIdx.x; e < E; e += kRouterThreads)
    s_load[e] = e < a.experts ? dloss * a.load[run.s * a.experts + e] : 0.0f;
  __syncthreads();
  float2 load[P];
#pragma unroll
  for (int i = 0; i < P; ++i) load[i] = reinterpret_cast<const float2*>(s_load + first)[i];
  T* const mine = s_row[warp * TPW + sub];
  const int64_t t0 = run.first + sub;
  const int tokens = static_cast<int>(run.end - run.first);
  for (int q = warp * TPW; q < tokens; q += kStep) {
    const bool in = q + sub < tokens;
    const int64_t t = t0 + q, at = t * a.top_k;
    const T* const row = static_cast<const T*>(a.logits) + t * a.ld;
    const bool live = in && (!a.mask || a.mask[t] != 0);
    const bool picks = live && a.dweights;
    // The lane's (first) choice: expert (-1: none) and dw.
    int e0 = -1;
    float d = 0.0f;
    if (picks && l < a.top_k) {
      e0 = a.indices[at + l];
      d = a.dweights[at + l];
    }
    float y[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) y[i] = -INFINITY;
    if (live) load_row<T, EPL>(row, first, a.experts, a.vec, y);
    if (static_cast<uint32_t>(e0) >= static_cast<uint32_t>(a.experts)) e0 = -1;
    const float x0 = e0 >= 0 ? to_f(row[e0]) : 0.0f;
    const float d0 = a.normalize ? __shfl_sync(kFull, d, lane - l) : 0.0f;
    d -= d0;
    // Choices past the lanes' first ones.
    auto choice = [&](int j, int& e, float& dw, float& logit) {
      e = a.indices[at + j];
      dw = a.dweights[at + j] - d0;
      if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(a.experts)) e = -1;
      logit = e >= 0 ? to_f(row[e]) : 0.0f;
    };
    float m = y[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, y[i]);
    m = group_max_f<LPT>(m);
    // A row of -inf alone (one left out, too): its exponentials are zero.
    const bool none = !(m > -INFINITY);
    if (none) m = 0.0f;
    float2 x[P], se = both(0.0f), sl = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 u = __fadd2_rn(make_float2(y[2 * i], y[2 * i + 1]), both(-m));
      x[i] = make_float2(exp_of(u.x), exp_of(u.y));
      se = __fadd2_rn(se, x[i]);
      sl = __ffma2_rn(x[i], load[i], sl);
    }
    float v[4] = {se.x + se.y, sl.x + sl.y, 0.0f, 0.0f};  // sum(e), sum(e load), z, s
    const float ex0 = e0 >= 0 ? exp_of(x0 - m) : 0.0f;
    v[2] = ex0;
    v[3] = e0 >= 0 ? ex0 * d : 0.0f;
    if (a.top_k > LPT && picks)
      for (int j = l + LPT; j < a.top_k; j += LPT) {
        int e;
        float dw, logit;
        choice(j, e, dw, logit);
        if (e >= 0) {
          const float ex = exp_of(logit - m);
          v[2] += ex;
          v[3] = fmaf(ex, dw, v[3]);
        }
      }
    group_sum4<LPT>(v);
    // Left out: masked, or no logit above -inf and no NaN (the sum would be one).
    const bool any = live && !(none && v[0] == 0.0f);
    const float inv = any ? __frcp_rn(v[0]) : 0.0f, base = v[1] * inv;
    const float dot = a.normalize ? base : fmaf(v[3], inv, base);
    // The row without its chosen ones' own gradients, p (load - dot) ...
    const float2 inv2 = both(inv), off = both(-dot * inv);
#pragma unroll
    for (int j = 0; j < EPL; j += W) {
      Vec16<T> o;
#pragma unroll
      for (int i = 0; i < W; i += 2)
        set_pair(&o.e[i], __fmul2_rn(x[(j + i) / 2], __ffma2_rn(load[(j + i) / 2], inv2, off)));
      *reinterpret_cast<Vec16<T>*>(mine + first + j) = o;
    }
    __syncwarp();
    // ... and those: p * (load + dp - dot), dp = dw, or (dw - s/z) sum/z.
    const float rz = __frcp_rn(v[2]), mean_d = v[3] * rz;
    auto put = [&](int e, float ex, float dw) {
      const float dp = a.normalize ? (dw - mean_d) * rz * v[0] : dw;
      from_f(mine[e], ex * inv * (s_load[e] + dp - dot));
    };
    if (any && e0 >= 0) put(e0, ex0, d);
    if (a.top_k > LPT && any && picks)
      for (int j = l + LPT; j < a.top_k; j += LPT) {
        int e;
        float dw, logit;
        choice(j, e, dw, logit);
        if (e >= 0) put(e, exp_of(logit - m), dw);
      }
    __syncwarp();
    if (in) {
      T* const out = static_cast<T*>(a.dlogits) + t * a.lddx + first;
      if (a.vec && first + EPL <= a.experts) {
#pragma unroll
        for (int j = 0; j < EPL; j += W)
          *reinterpret_cast<Vec16<T>*>(out + j) = *reinterpret_cast<const Vec16<T>*>(mine + first + j);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (first + i < a.experts) out[i] = mine[first + i];
      }
    }
    __syncwarp();
  }
}

template <typename T, int LPT, int EPL>
mx_status run_cfg(const RouterArgs& a, int64_t ctas, bool backward, cudaStream_t s) {
  auto kern = backward ? router_backward_kernel<T, LPT, EPL> : router_forward_kernel<T, LPT, EPL>;
  return cuda_status(launch_kernel(kern, static_cast<unsigned>(ctas), kRouterThreads, 0, s, 1, a), "mx_router launch");
}

// Lanes a token by the number of experts, eight experts a lane (sixteen above 256).
// Half the lanes with sixteen each: the backward pass of 65536 tokens took 32.2
// instead of 30.2 us with 256 experts, 16.0 instead of 11.0 with 64 (twice the
// registers, half the warps).
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
  int width = 32;
  while (width < L.experts) width *= 2;
  // One launch where eight CTAs are enough for the sequences: the same time on
  // the device (8.5 us in all for 256 tokens), and a call on the host takes 27 us
  // instead of 30, which is what bounds it up to some 100000 tokens.
  if (p.seqs <= kTailSeqs)
    return cuda_status(launch_kernel(router_tail_kernel, kTailCtas, 1024, 0, s, kTailCtas, q, width),
                       "mx_router launch (sums)");
  st = cuda_status(launch_kernel(router_sequence_kernel, static_cast<unsigned>(p.seqs), 1024, 0, s, 1, q),
                   "mx_router launch (sequences)");
  if (st != MX_OK) return st;
  const int64_t grid = std::min<int64_t>(sm_count(), (p.seqs * width + 8191) / 8192);
  return cuda_status(launch_kernel(router_finish_kernel, static_cast<unsigned>(grid), 1024, 0, s, 1, q, width),
                     "mx_router launch (loss)");
}

mx_status launch_router_backward(const RouterLaunch& L, cudaStream_t s) {
  const RouterPlan p = router_plan(L.tokens, L.tokens_per_seq, L.experts, kBackwardCtas, kRouterWarps);
  const RouterArgs a = router_args(L, p);
  return L.dtype == MX_F32 ? run_any<float>(a, p.ctas(), true, s) : run_any<__nv_bfloat16>(a, p.ctas(), true, s);
}

}  // namespace mx
