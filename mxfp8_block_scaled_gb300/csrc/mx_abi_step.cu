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

// The copies that `axis` asks for of a [rows, cols] matrix: present and aligned,
// sizes whole blocks (mx_quantize's rules).
mx_status check_copies(const char* fn, int axis, int64_t rows, int64_t cols, const void* row_data, const void* row_scale,
                       const void* col_data, const void* col_scale, bool grouped) {
  const bool row = (axis & MX_ROWWISE) != 0, col = (axis & MX_COLWISE) != 0;
  if (cols % 32 != 0 || (col && !grouped && rows % 32 != 0)) {
    set_error("%s: the columns (and the rows for a dense column copy) must be a multiple of 32", fn);
    return MX_ERR_UNSUPPORTED_SHAPE;
  }
  if (rows == 0 || cols == 0) return MX_OK;
  if ((row && (!row_data || !row_scale)) || (col && (!col_data || !col_scale))) {
    set_error("%s: a requested copy is null", fn);
    return MX_ERR_INVALID_ARG;
  }
  for (const void* p : {row_data, row_scale, col_data, col_scale}) {
    if (!aligned(p, 16)) {
      set_error("%s: the copies must be 16-byte aligned", fn);
      return MX_ERR_ALIGNMENT;
    }
  }
  return MX_OK;
}

// A matrix that is read or written in 16-byte pieces.
mx_status check_wide_matrix(const char* fn, const char* name, const void* p, int64_t ld, int64_t cols, int elem) {
  if (!p || ld < cols) {
    set_error("%s: %s is null or its pitch is less than its columns", fn, name);
    return MX_ERR_INVALID_ARG;
  }
  if (!aligned(p, 16) || ld % (16 / elem) != 0) {
    set_error("%s: %s and its rows must be 16-byte aligned", fn, name);
    return MX_ERR_ALIGNMENT;
  }
  return MX_OK;
}

// What both directions of the norm with the residual's addition share.
mx_status check_add_norm(const char* fn, int64_t rows, int64_t cols, int stream_dtype, int param_dtype, int axis) {
  if (rows < 0 || cols < 1 || !known_dtype(stream_dtype) || !known_dtype(param_dtype) || axis < 0 || axis > MX_BOTH) {
    set_error("%s: needs rows >= 0, cols >= 1, a known stream_dtype and param_dtype, axis 0 or an mx_axis", fn);
    return MX_ERR_INVALID_ARG;
  }
  if (cols > MX_ADD_NORM_MAX_COLS || rows > 0x7FFFFFFFLL) {
    set_error("%s: at most %d columns and 2^31 - 1 rows", fn, MX_ADD_NORM_MAX_COLS);
    return MX_ERR_UNSUPPORTED_SHAPE;
  }
  return MX_OK;
}

#define MX_CHECK(call)                       \
  do {                                       \
    const mx_status check_st = (call);       \
    if (check_st != MX_OK) return check_st;  \
  } while (0)

// Both directions of the gate.
mx_status gated(const char* fn, bool backward, const void* dh, int64_t lddh, const void* gate_up, int64_t ld, int64_t rows,
                int64_t f, int act, int axis, void* row_data, void* row_scale, void* col_data, void* col_scale,
                const int64_t* group_offsets, int n_groups, int64_t col_capacity, int* dev_status, void* stream) {
  if (rows < 0 || f < 0 || act < MX_ACT_NONE || act > MX_ACT_SILU || axis < MX_ROWWISE || axis > MX_BOTH) {
    set_error("%s: negative size, unknown act %d or axis %d", fn, act, axis);
    return MX_ERR_INVALID_ARG;
  }
  if (rows > 0x7FFFFFFFLL || f > 0x3FFFFFFFLL) {
    set_error("%s: rows must be < 2^31, F < 2^30", fn);
    return MX_ERR_UNSUPPORTED_SHAPE;
  }
  const bool grouped = group_offsets != nullptr, col = (axis & MX_COLWISE) != 0;
  MX_CHECK(check_copies(fn, axis, rows, f, row_data, row_scale, col_data, col_scale, grouped));
  if (grouped) {
    if (n_groups < 1 || (col && (col_capacity < 0 || col_capacity % 128 != 0))) {
      set_error("%s: needs n_groups >= 1 and col_capacity a multiple of 128", fn);
      return MX_ERR_INVALID_ARG;
    }
    if (n_groups > MX_MAX_GROUPS || col_capacity > 0x7FFFFFFFLL) {
      set_error("%s: at most %d groups, col_capacity < 2^31", fn, MX_MAX_GROUPS);
      return MX_ERR_UNSUPPORTED_SHAPE;
    }
    MX_CHECK(check_aligned(fn, "group_offsets", group_offsets, 8));
  }
  if (rows == 0 || f == 0) return MX_OK;
  if (grouped && col && col_capacity == 0) {  // the kernel would refuse it, unseen without a dev_status
    set_error("%s: col_capacity is 0 but rows > 0", fn);
    return MX_ERR_UNSUPPORTED_SHAPE;
  }
  if (backward) MX_CHECK(check_wide_matrix(fn, "dh", dh, lddh, f, 2));
  MX_CHECK(check_wide_matrix(fn, "gate_up", gate_up, ld, 2 * f, 2));
  MX_CHECK(check_device());
  GatedLaunch L = {};
  L.dh = backward ? dh : nullptr;
  L.lddh = lddh;
  L.gate_up = gate_up;
  L.ld = ld;
  L.rows = rows;
  L.f = f;
  L.act = act;
  if (axis & MX_ROWWISE) {
    L.row_data = row_data;
    L.row_scale = row_scale;
  }
  if (col) {
    L.col_data = col_data;
    L.col_scale = col_scale;
  }
  if (grouped && col) {  // a row copy has no segments
    L.offsets = group_offsets;
    L.n_groups = n_groups;
  }
  L.col_pitch = grouped ? col_capacity : rows;
  L.dev_status = dev_status;
  return launch_gated(L, static_cast<cudaStream_t>(stream));
}

thread_local WaitTest g_wait_test = {};

}  // namespace

mx::WaitTest mx::take_wait_test() {
  const WaitTest t = g_wait_test;
  g_wait_test = WaitTest{};
  return t;
}

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

mx_status mx_selftest_block_timeout(int what, uint64_t timeout_ns) {
  if (what < 0 || what > 2 || (what != 0 && (timeout_ns < 1000000ull || timeout_ns > 10000000000ull))) {
    set_error("mx_selftest_block_timeout: needs what 0, 1 or 2, 1 ms <= timeout_ns <= 10 s");
    return MX_ERR_INVALID_ARG;
  }
  g_wait_test = WaitTest{what, timeout_ns};
  return MX_OK;
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

mx_status mx_add_norm_quantize(const void* x, int64_t ldx, const void* residual, int64_t ld_residual, int stream_dtype,
                               const void* weight, int param_dtype, int64_t rows, int64_t cols, float eps, int axis,
                               void* sum, int64_t ld_sum, void* y, int64_t ldy, float* rstd, void* row_data,
                               void* row_scale, void* col_data, void* col_scale, int* dev_status, void* stream) {
  const char* fn = "mx_add_norm_quantize";
  MX_CHECK(check_add_norm(fn, rows, cols, stream_dtype, param_dtype, axis));
  if (!(eps >= 0.0f) || !std::isfinite(eps)) {
    set_error("mx_add_norm_quantize: eps must be finite and not negative");
    return MX_ERR_INVALID_ARG;
  }
  if (axis == 0 && !y && rows > 0) {
    set_error("mx_add_norm_quantize: axis 0 without y: nothing of the norm's output is wanted");
    return MX_ERR_INVALID_ARG;
  }
  MX_CHECK(check_copies(fn, axis, rows, cols, row_data, row_scale, col_data, col_scale, false));
  if (rows == 0) return MX_OK;
  const int elem = elem_size(stream_dtype);
  MX_CHECK(check_wide_matrix(fn, "x", x, ldx, cols, 2));
  if (residual) MX_CHECK(check_wide_matrix(fn, "residual", residual, ld_residual, cols, elem));
  if (sum) MX_CHECK(check_wide_matrix(fn, "sum", sum, ld_sum, cols, elem));
  if (y) MX_CHECK(check_wide_matrix(fn, "y", y, ldy, cols, 2));
  MX_CHECK(check_aligned(fn, "weight", weight, elem_size(param_dtype)));
  MX_CHECK(check_aligned(fn, "rstd", rstd, 4));
  MX_CHECK(check_device());
  AddNormLaunch L = {};
  L.stream_f32 = stream_dtype == MX_F32;
  L.first = x;
  L.ld_first = ldx;
  L.second = residual;
  L.ld_second = ld_residual;
  L.weight = weight;
  L.param_dtype = param_dtype;
  L.rows = rows;
  L.cols = cols;
  L.eps = eps;
  L.out = sum;
  L.ld_out = ld_sum;
  L.y = y;
  L.ldy = ldy;
  L.rstd = rstd;
  if (axis & MX_ROWWISE) {
    L.row_data = row_data;
    L.row_scale = row_scale;
  }
  if (axis & MX_COLWISE) {
    L.col_data = col_data;
    L.col_scale = col_scale;
  }
  L.dev_status = dev_status;
  return launch_add_norm(L, static_cast<cudaStream_t>(stream));
}

size_t mx_add_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  return rows <= 0 || cols <= 0 ? 0 : add_norm_backward_workspace(rows, cols);
}

mx_status mx_add_norm_backward(const void* dy, int64_t lddy, const void* sum, int64_t ld_sum, const void* dsum,
                               int64_t ld_dsum, int stream_dtype, const void* weight, int param_dtype,
                               const float* rstd, int64_t rows, int64_t cols, int axis, void* dx, int64_t lddx,
                               float* dweight, void* row_data, void* row_scale, void* col_data, void* col_scale,
                               void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  const char* fn = "mx_add_norm_backward";
  MX_CHECK(check_add_norm(fn, rows, cols, stream_dtype, param_dtype, axis));
  MX_CHECK(check_copies(fn, axis, rows, cols, row_data, row_scale, col_data, col_scale, false));
  MX_CHECK(check_aligned(fn, "dweight", dweight, 4));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (!dweight) return MX_OK;
    MX_CHECK(check_device());
    return cuda_status(cudaMemsetAsync(dweight, 0, static_cast<size_t>(cols) * 4, s), "cudaMemsetAsync");
  }
  const int elem = elem_size(stream_dtype);
  MX_CHECK(check_wide_matrix(fn, "dy", dy, lddy, cols, 2));
  MX_CHECK(check_wide_matrix(fn, "sum", sum, ld_sum, cols, elem));
  if (dsum) MX_CHECK(check_wide_matrix(fn, "dsum", dsum, ld_dsum, cols, elem));
  if (dx || axis == 0) MX_CHECK(check_wide_matrix(fn, "dx", dx, lddx, cols, elem));
  MX_CHECK(check_present(fn, "rstd", rstd, 4));
  MX_CHECK(check_aligned(fn, "weight", weight, elem_size(param_dtype)));
  if (dweight) MX_CHECK(check_workspace(fn, workspace, workspace_bytes, add_norm_backward_workspace(rows, cols)));
  MX_CHECK(check_device());
  AddNormLaunch L = {};
  L.backward = true;
  L.stream_f32 = stream_dtype == MX_F32;
  L.first = dy;
  L.ld_first = lddy;
  L.second = sum;
  L.ld_second = ld_sum;
  L.third = dsum;
  L.ld_third = ld_dsum;
  L.weight = weight;
  L.param_dtype = param_dtype;
  L.rows = rows;
  L.cols = cols;
  L.out = dx;
  L.ld_out = lddx;
  L.rstd = const_cast<float*>(rstd);
  if (axis & MX_ROWWISE) {
    L.row_data = row_data;
    L.row_scale = row_scale;
  }
  if (axis & MX_COLWISE) {
    L.col_data = col_data;
    L.col_scale = col_scale;
  }
  L.dweight = dweight;
  L.ws = workspace;
  L.dev_status = dev_status;
  return launch_add_norm(L, s);
}

mx_status mx_gated_quantize(const void* gate_up, int64_t ld, int64_t rows, int64_t f, int act, int axis, void* row_data,
                            void* row_scale, void* col_data, void* col_scale, const int64_t* group_offsets, int n_groups,
                            int64_t col_capacity, int* dev_status, void* stream) {
  return gated("mx_gated_quantize", false, nullptr, 0, gate_up, ld, rows, f, act, axis, row_data, row_scale, col_data,
               col_scale, group_offsets, n_groups, col_capacity, dev_status, stream);
}

mx_status mx_gated_backward_quantize(const void* dh, int64_t lddh, const void* gate_up, int64_t ld, int64_t rows,
                                     int64_t f, int act, int axis, void* row_data, void* row_scale, void* col_data,
                                     void* col_scale, const int64_t* group_offsets, int n_groups, int64_t col_capacity,
                                     int* dev_status, void* stream) {
  return gated("mx_gated_backward_quantize", true, dh, lddh, gate_up, ld, rows, f, act, axis, row_data, row_scale,
               col_data, col_scale, group_offsets, n_groups, col_capacity, dev_status, stream);
}

}  // extern "C"
