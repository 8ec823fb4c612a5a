// mx_abi_step.cu - the C ABI of the operators around the products of a
// training step (include/mxfp8.h): host-side validation and dispatch on the
// caller's stream. No device memory is allocated here.

#include <cuda_runtime.h>

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

}  // extern "C"
