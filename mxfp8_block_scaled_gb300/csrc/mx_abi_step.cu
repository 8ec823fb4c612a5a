// mx_abi_step.cu - the C ABI of the operators around the products of a
// training step (include/mxfp8.h): host-side validation and dispatch on the
// caller's stream. No device memory is allocated here.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "mx_internal.h"

using namespace mx;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool known_dtype(int dtype) { return dtype == MX_BF16 || dtype == MX_F32; }

int elem_size(int dtype) { return dtype == MX_F32 ? 4 : 2; }

mx_status check_adamw_tensor(const mx_adamw_tensor& t, int i, int bits) {
  if (t.numel < 0 || t.reserved != 0 || !known_dtype(t.grad_dtype) || !std::isfinite(t.weight_decay)) {
    set_error("mx_adamw_step: tensor %d: negative numel, reserved field set, unknown grad_dtype or weight_decay not finite",
              i);
    return MX_ERR_INVALID_ARG;
  }
  if (t.numel == 0) return MX_OK;
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq ||
      (bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale))) {
    set_error("mx_adamw_step: tensor %d: null pointer", i);
    return MX_ERR_INVALID_ARG;
  }
  const bool states = bits == 8 ? aligned(t.exp_avg_scale, 4) && aligned(t.exp_avg_sq_scale, 4)
                                : aligned(t.exp_avg, 4) && aligned(t.exp_avg_sq, 4);
  if (!aligned(t.param, 4) || !aligned(t.grad, elem_size(t.grad_dtype)) || !states) {
    set_error("mx_adamw_step: tensor %d: a pointer is not aligned to its element type", i);
    return MX_ERR_ALIGNMENT;
  }
  return MX_OK;
}

// Sizes, types and pitches that both directions of the norm share.
mx_status check_norm(const char* fn, int64_t rows, int64_t cols, int dtype, int param_dtype, int center) {
  if (rows < 0 || cols < 1 || !known_dtype(dtype) || !known_dtype(param_dtype) || (center != 0 && center != 1)) {
    set_error("%s: needs rows >= 0, cols >= 1, a known dtype and param_dtype, center 0 or 1", fn);
    return MX_ERR_INVALID_ARG;
  }
  if (cols > 0x7FFFFFFFLL) {
    set_error("%s: cols must be < 2^31", fn);
    return MX_ERR_UNSUPPORTED_SHAPE;
  }
  return MX_OK;
}

// A matrix argument: present, a pitch of at least cols, aligned to its type.
mx_status check_matrix(const char* fn, const char* name, const void* p, int64_t ld, int64_t cols, int elem) {
  if (!p || ld < cols) {
    set_error("%s: %s is null or its pitch is less than its columns", fn, name);
    return MX_ERR_INVALID_ARG;
  }
  if (!aligned(p, elem)) {
    set_error("%s: %s is not aligned to its element type", fn, name);
    return MX_ERR_ALIGNMENT;
  }
  return MX_OK;
}

mx_status check_aligned(const char* fn, const char* name, const void* p, int a) {
  if (aligned(p, a)) return MX_OK;
  set_error("%s: %s is not %d-byte aligned", fn, name, a);
  return MX_ERR_ALIGNMENT;
}

// Scratch of at least `need` bytes, 16-byte aligned.
mx_status check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need) {
    set_error("%s: needs a workspace of %llu bytes", fn, static_cast<unsigned long long>(need));
    return MX_ERR_INVALID_ARG;
  }
  return check_aligned(fn, "workspace", ws, 16);
}

// Tokens of a sequence, as the router's sizes are computed from them: `tokens` or
// more are one sequence (their sums could pass 64 bits).
int64_t sequence_tokens(int64_t tokens_per_seq, int64_t tokens) {
  return std::min(tokens_per_seq, std::max<int64_t>(tokens, 1));
}

// What both directions of the router share; MX_OK with tokens = 0 too.
mx_status check_router(const char* fn, int dtype, int64_t tokens, int64_t tokens_per_seq, int experts, int top_k,
                       int normalize) {
  if (!known_dtype(dtype) || tokens < 0 || tokens_per_seq < 1 || experts < 1 || top_k < 1 || top_k > experts ||
      (normalize != 0 && normalize != 1)) {
    set_error("%s: needs a known dtype, tokens >= 0, tokens_per_seq >= 1, 1 <= top_k <= experts, normalize 0 or 1", fn);
    return MX_ERR_INVALID_ARG;
  }
  if (experts > MX_MAX_GROUPS || tokens > 0x7FFFFFFFLL || (tokens > 0 && !router_fits(tokens, tokens_per_seq, experts))) {
    set_error("%s: at most %d experts and 2^31 - 1 tokens", fn, MX_MAX_GROUPS);
    return MX_ERR_UNSUPPORTED_SHAPE;
  }
  return MX_OK;
}

mx_status check_present(const char* fn, const char* name, const void* p, int a) {
  if (!p) {
    set_error("%s: %s is null", fn, name);
    return MX_ERR_INVALID_ARG;
  }
  return check_aligned(fn, name, p, a);
}

#define MX_CHECK(call)                       \
  do {                                       \
    const mx_status check_st = (call);       \
    if (check_st != MX_OK) return check_st;  \
  } while (0)

}  // namespace

extern "C" {

mx_status mx_adamw_step(const mx_adamw_tensor* tensors, int n, int state_bits, const mx_adamw_hyper* hyper,
                        const float* grad_scale, int* dev_status, void* stream) {
  if (n < 0 || (n > 0 && !tensors) || !hyper) {
    set_error("mx_adamw_step: null tensors or hyper, or negative n");
    return MX_ERR_INVALID_ARG;
  }
  if (state_bits != 32 && state_bits != 8) {
    set_error("mx_adamw_step: state_bits must be 32 or 8, got %d", state_bits);
    return MX_ERR_INVALID_ARG;
  }
  const mx_adamw_hyper& h = *hyper;
  if (!std::isfinite(h.lr) || !(h.beta1 >= 0.0 && h.beta1 < 1.0) || !(h.beta2 >= 0.0 && h.beta2 < 1.0) ||
      !(h.eps >= 0.0) || !std::isfinite(h.eps) || h.step < 1 || h.reserved != 0) {
    set_error("mx_adamw_step: needs lr finite, 0 <= beta < 1, eps >= 0, step >= 1 and reserved = 0");
    return MX_ERR_INVALID_ARG;
  }
  if (!aligned(grad_scale, 4)) {
    set_error("mx_adamw_step: grad_scale is not 4-byte aligned");
    return MX_ERR_ALIGNMENT;
  }
  for (int i = 0; i < n; ++i) {
    const mx_status st = check_adamw_tensor(tensors[i], i, state_bits);
    if (st != MX_OK) return st;
  }
  if (n == 0) return MX_OK;
  const mx_status st = check_device();
  if (st != MX_OK) return st;
  return launch_adamw(tensors, n, state_bits, h, grad_scale, dev_status, static_cast<cudaStream_t>(stream));
}

mx_status mx_layer_norm(const void* x, int64_t ldx, const void* weight, const void* bias, int param_dtype, int64_t rows,
                        int64_t cols, float eps, int center, int dtype, void* y, int64_t ldy, float* mean, float* rstd,
                        int* dev_status, void* stream) {
  const char* fn = "mx_layer_norm";
  MX_CHECK(check_norm(fn, rows, cols, dtype, param_dtype, center));
  if (!(eps >= 0.0f) || !std::isfinite(eps)) {
    set_error("mx_layer_norm: eps must be finite and not negative");
    return MX_ERR_INVALID_ARG;
  }
  if (rows == 0) return MX_OK;
  MX_CHECK(check_matrix(fn, "x", x, ldx, cols, elem_size(dtype)));
  MX_CHECK(check_matrix(fn, "y", y, ldy, cols, elem_size(dtype)));
  MX_CHECK(check_aligned(fn, "weight", weight, elem_size(param_dtype)));
  MX_CHECK(check_aligned(fn, "bias", bias, elem_size(param_dtype)));
  MX_CHECK(check_aligned(fn, "mean", mean, 4));
  MX_CHECK(check_aligned(fn, "rstd", rstd, 4));
  MX_CHECK(check_device());
  NormLaunch L = {};
  L.x = x;
  L.ldx = ldx;
  L.weight = weight;
  L.bias = bias;
  L.param_dtype = param_dtype;
  L.rows = rows;
  L.cols = cols;
  L.dtype = dtype;
  L.center = center;
  L.eps = eps;
  L.out = y;
  L.ldo = ldy;
  L.mean = mean;
  L.rstd = rstd;
  L.dev_status = dev_status;
  return launch_norm_forward(L, static_cast<cudaStream_t>(stream));
}

size_t mx_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  return rows <= 0 || cols <= 0 ? 0 : norm_backward_workspace(rows, cols);
}

mx_status mx_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight,
                                 int param_dtype, const float* mean, const float* rstd, int64_t rows, int64_t cols,
                                 int center, int dtype, void* dx, int64_t lddx, float* dweight, float* dbias,
                                 void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  const char* fn = "mx_layer_norm_backward";
  MX_CHECK(check_norm(fn, rows, cols, dtype, param_dtype, center));
  MX_CHECK(check_aligned(fn, "dweight", dweight, 4));
  MX_CHECK(check_aligned(fn, "dbias", dbias, 4));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (!dweight && !dbias) return MX_OK;
    MX_CHECK(check_device());
    for (float* p : {dweight, dbias})
      if (p) MX_CHECK(cuda_status(cudaMemsetAsync(p, 0, static_cast<size_t>(cols) * 4, s), "cudaMemsetAsync"));
    return MX_OK;
  }
  const int elem = elem_size(dtype);
  MX_CHECK(check_matrix(fn, "dy", dy, lddy, cols, elem));
  MX_CHECK(check_matrix(fn, "x", x, ldx, cols, elem));
  MX_CHECK(check_matrix(fn, "dx", dx, lddx, cols, elem));
  if (!rstd || (center && !mean)) {
    set_error("mx_layer_norm_backward: null rstd or mean");
    return MX_ERR_INVALID_ARG;
  }
  MX_CHECK(check_aligned(fn, "weight", weight, elem_size(param_dtype)));
  MX_CHECK(check_aligned(fn, "mean", mean, 4));
  MX_CHECK(check_aligned(fn, "rstd", rstd, 4));
  if (dweight || dbias) MX_CHECK(check_workspace(fn, workspace, workspace_bytes, norm_backward_workspace(rows, cols)));
  MX_CHECK(check_device());
  NormLaunch L = {};
  L.x = x;
  L.ldx = ldx;
  L.dy = dy;
  L.lddy = lddy;
  L.weight = weight;
  L.param_dtype = param_dtype;
  L.rows = rows;
  L.cols = cols;
  L.dtype = dtype;
  L.center = center;
  L.out = dx;
  L.ldo = lddx;
  L.mean = const_cast<float*>(mean);
  L.rstd = const_cast<float*>(rstd);
  L.dweight = dweight;
  L.dbias = dbias;
  L.ws = workspace;
  L.dev_status = dev_status;
  return launch_norm_backward(L, s);
}

mx_status mx_selftest_norm_timeout(uint64_t timeout_ns, const void* dy, const void* x, int64_t rows, int64_t cols,
                                   void* out, float* rstd, float* dweight, float* dbias, void* workspace,
                                   size_t workspace_bytes, int* dev_status, void* stream) {
  const char* fn = "mx_selftest_norm_timeout";
  if (timeout_ns < 1000000ull || timeout_ns > 10000000000ull || rows < 1 || cols < 257 || cols > 16384) {
    set_error("mx_selftest_norm_timeout: needs 1 ms <= timeout_ns <= 10 s, rows >= 1, 257 <= cols <= 16384");
    return MX_ERR_INVALID_ARG;
  }
  if (dy) MX_CHECK(check_matrix(fn, "dy", dy, cols, cols, 2));
  MX_CHECK(check_matrix(fn, "x", x, cols, cols, 2));
  MX_CHECK(check_matrix(fn, "out", out, cols, cols, 2));
  MX_CHECK(check_present(fn, "rstd", rstd, 4));
  if (dy) {
    MX_CHECK(check_present(fn, "dweight", dweight, 4));
    MX_CHECK(check_present(fn, "dbias", dbias, 4));
    MX_CHECK(check_workspace(fn, workspace, workspace_bytes, norm_backward_workspace(rows, cols)));
  }
  MX_CHECK(check_device());
  NormLaunch L = {};
  L.x = x;
  L.ldx = cols;
  L.dy = dy;
  L.lddy = cols;
  L.param_dtype = MX_F32;
  L.rows = rows;
  L.cols = cols;
  L.dtype = MX_BF16;
  L.eps = 1e-5f;
  L.out = out;
  L.ldo = cols;
  L.rstd = rstd;
  L.dweight = dweight;
  L.dbias = dbias;
  L.ws = workspace;
  L.dev_status = dev_status;
  L.timeout_ns = timeout_ns;
  L.withheld = 16;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dy ? launch_norm_backward(L, s) : launch_norm_forward(L, s);
}

size_t mx_epilogue_backward_workspace_bytes(int64_t rows, int64_t cols) {
  return rows <= 0 || cols <= 0 ? 0 : epilogue_backward_workspace(rows, cols);
}

mx_status mx_epilogue_backward(const void* dy, int64_t lddy, const void* preact, int64_t ld_preact, int64_t rows,
                               int64_t cols, int act, void* dz, int64_t lddz, float* dbias, void* workspace,
                               size_t workspace_bytes, int* dev_status, void* stream) {
  const char* fn = "mx_epilogue_backward";
  (void)dev_status;
  if (rows < 0 || cols < 0 || act < MX_ACT_NONE || act > MX_ACT_SILU) {
    set_error("mx_epilogue_backward: negative size or unknown act %d", act);
    return MX_ERR_INVALID_ARG;
  }
  if (rows > 0x7FFFFFFFLL || cols > 0x7FFFFFFFLL) {
    set_error("mx_epilogue_backward: sizes must be < 2^31");
    return MX_ERR_UNSUPPORTED_SHAPE;
  }
  MX_CHECK(check_aligned(fn, "dbias", dbias, 4));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cols == 0 || (!dz && !dbias)) return MX_OK;
  if (rows == 0) {
    if (!dbias) return MX_OK;
    MX_CHECK(check_device());
    return cuda_status(cudaMemsetAsync(dbias, 0, static_cast<size_t>(cols) * 4, s), "cudaMemsetAsync");
  }
  MX_CHECK(check_matrix(fn, "dy", dy, lddy, cols, 2));
  if (act != MX_ACT_NONE) MX_CHECK(check_matrix(fn, "preact", preact, ld_preact, cols, 2));
  if (dz) MX_CHECK(check_matrix(fn, "dz", dz, lddz, cols, 2));
  const size_t need = epilogue_backward_workspace(rows, cols);
  if (dbias && need > 0) MX_CHECK(check_workspace(fn, workspace, workspace_bytes, need));
  MX_CHECK(check_device());
  EpilogueBackwardLaunch L = {};
  L.dy = dy;
  L.lddy = lddy;
  L.z = preact;
  L.ldz = ld_preact;
  L.rows = rows;
  L.cols = cols;
  L.act = act;
  L.dz = dz;
  L.lddz = lddz;
  L.dbias = dbias;
  L.ws = workspace;
  return launch_epilogue_backward(L, s);
}

size_t mx_router_workspace_bytes(int64_t tokens, int64_t tokens_per_seq, int n_experts) {
  if (tokens <= 0 || tokens_per_seq <= 0 || n_experts <= 0) return 0;
  return router_workspace(tokens, sequence_tokens(tokens_per_seq, tokens), n_experts);
}

mx_status mx_router_forward(const void* logits, int64_t ld, int dtype, const uint8_t* token_mask, int64_t tokens,
                            int64_t tokens_per_seq, int n_experts, int top_k, int normalize, float coef,
                            int32_t* indices, float* weights, int64_t* counts, int64_t* group_offsets, float* load,
                            float* loss, void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  const char* fn = "mx_router_forward";
  (void)dev_status;
  tokens_per_seq = sequence_tokens(tokens_per_seq, tokens);
  MX_CHECK(check_router(fn, dtype, tokens, tokens_per_seq, n_experts, top_k, normalize));
  if (!std::isfinite(coef)) {
    set_error("mx_router_forward: coef is not finite");
    return MX_ERR_INVALID_ARG;
  }
  MX_CHECK(check_present(fn, "counts", counts, 8));
  MX_CHECK(check_present(fn, "group_offsets", group_offsets, 8));
  MX_CHECK(check_present(fn, "loss", loss, 4));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    MX_CHECK(check_device());
    MX_CHECK(cuda_status(cudaMemsetAsync(counts, 0, static_cast<size_t>(n_experts) * 8, s), "cudaMemsetAsync"));
    MX_CHECK(cuda_status(cudaMemsetAsync(group_offsets, 0, static_cast<size_t>(n_experts + 1) * 8, s), "cudaMemsetAsync"));
    return cuda_status(cudaMemsetAsync(loss, 0, 4, s), "cudaMemsetAsync");
  }
  MX_CHECK(check_matrix(fn, "logits", logits, ld, n_experts, elem_size(dtype)));
  MX_CHECK(check_present(fn, "indices", indices, 4));
  MX_CHECK(check_present(fn, "weights", weights, 4));
  MX_CHECK(check_present(fn, "load", load, 4));
  MX_CHECK(check_workspace(fn, workspace, workspace_bytes, router_workspace(tokens, tokens_per_seq, n_experts)));
  MX_CHECK(check_device());
  RouterLaunch L = {};
  L.logits = logits;
  L.ld = ld;
  L.dtype = dtype;
  L.mask = token_mask;
  L.tokens = tokens;
  L.tokens_per_seq = tokens_per_seq;
  L.experts = n_experts;
  L.top_k = top_k;
  L.normalize = normalize;
  L.coef = coef;
  L.indices = indices;
  L.weights = weights;
  L.counts = counts;
  L.offsets = group_offsets;
  L.load = load;
  L.loss = loss;
  L.ws = workspace;
  return launch_router_forward(L, s);
}

mx_status mx_router_backward(const void* logits, int64_t ld, int dtype, const uint8_t* token_mask, int64_t tokens,
                             int64_t tokens_per_seq, int n_experts, int top_k, int normalize, const int32_t* indices,
                             const float* load, const float* dweights, const float* dloss, void* dlogits, int64_t lddx,
                             int* dev_status, void* stream) {
  const char* fn = "mx_router_backward";
  (void)dev_status;
  tokens_per_seq = sequence_tokens(tokens_per_seq, tokens);
  MX_CHECK(check_router(fn, dtype, tokens, tokens_per_seq, n_experts, top_k, normalize));
  if (tokens == 0) return MX_OK;
  MX_CHECK(check_matrix(fn, "logits", logits, ld, n_experts, elem_size(dtype)));
  MX_CHECK(check_matrix(fn, "dlogits", dlogits, lddx, n_experts, elem_size(dtype)));
  MX_CHECK(check_present(fn, "load", load, 4));
  if (dweights) MX_CHECK(check_present(fn, "indices", indices, 4));
  MX_CHECK(check_aligned(fn, "dweights", dweights, 4));
  MX_CHECK(check_aligned(fn, "dloss", dloss, 4));
  MX_CHECK(check_device());
  RouterLaunch L = {};
  L.logits = logits;
  L.ld = ld;
  L.dtype = dtype;
  L.mask = token_mask;
  L.tokens = tokens;
  L.tokens_per_seq = tokens_per_seq;
  L.experts = n_experts;
  L.top_k = top_k;
  L.normalize = normalize;
  L.indices = const_cast<int32_t*>(indices);
  L.load = const_cast<float*>(load);
  L.dweights = dweights;
  L.dloss = dloss;
  L.dlogits = dlogits;
  L.lddx = lddx;
  return launch_router_backward(L, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
