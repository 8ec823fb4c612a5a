// mx_internal.h - declarations shared by the translation units of the library
// (host side only; no device code here).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <cstring>
#include <utility>

#include "../../include/mxfp8.h"

namespace mx {

// Last error message of this host thread (returned by mx_last_error()).
void set_error(const char* fmt, ...);

// MX_OK if e == cudaSuccess, else records the message and returns MX_ERR_CUDA.
mx_status cuda_status(cudaError_t e, const char* what);

// MX_OK if the current device is an sm_103 part (the kernels are built for
// sm_103a only).
mx_status check_device();

// Bounded-wait limit (nanoseconds) for device-side mbarrier waits. Read once
// from the MXFP8_WAIT_TIMEOUT_NS environment variable (default 2 s).
uint64_t wait_timeout_ns();

// What mx_selftest_block_timeout asked of the calling thread's next launch of the
// gated block's kernels, handed out once: which wait runs out (0: none), after how long.
struct WaitTest {
  int what;
  uint64_t timeout_ns;
  bool stages() const { return what == 1; }
  bool sums() const { return what == 2; }
  uint64_t limit() const { return what ? timeout_ns : wait_timeout_ns(); }
};
WaitTest take_wait_test();

// Number of SMs of the current device (cached per device).
int sm_count();

// Programmatic dependent launch on (default); MXFP8_PDL=0 turns it off.
bool pdl_enabled();

// Launches kern on stream s. With programmatic stream serialization the grid
// may be scheduled while the kernel before it on the stream is finishing; each
// kernel of this library runs griddepcontrol.wait before its first global
// memory access, which returns once that previous grid has completed and its
// writes are visible, and griddepcontrol.launch_dependents at its start (but for
// a sum of partial rows that holds the next kernel back, launch_column_reduce).
// cluster_x > 1 also sets the cluster shape.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                          unsigned cluster_x, Args&&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  std::memset(attr, 0, sizeof(attr));
  unsigned n = 0;
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// --- quantiser -------------------------------------------------------------
struct QuantLaunch {
  const void* x;
  int64_t rows, cols, ldx;
  void* row_data;
  void* row_scale;
  void* col_data;
  void* col_scale;
  const int64_t* offsets;  // nullptr: dense column copy
  int n_groups;
  int64_t col_pitch;       // rows (dense) or the grouped capacity
  int64_t batch;           // stacked matrices (1 unless batched)
  int64_t x_batch_stride;  // elements between stacked inputs
  bool x_f32 = false;      // FP32 input (else BF16)
  int* dev_status;
};
mx_status launch_quantize(const QuantLaunch& q, bool do_row, bool do_col, cudaStream_t s);
// Several dense BF16 matrices (batch 1 each, no groups) in one launch.
mx_status launch_quantize_multi(const QuantLaunch* qs, int n, bool do_row, bool do_col, cudaStream_t s);
// Current scaling: amax of each matrix of the stack q (zeroed first, then
// reduced), and the quantisation with scale[b] = amax[b] / format_max (1 for an
// invalid amax), written to `scale`.
mx_status launch_current_amax(const QuantLaunch& q, float* amax, cudaStream_t s);
mx_status launch_quantize_current(const QuantLaunch& q, const float* amax, float format_max, float* scale,
                                  bool do_row, bool do_col, cudaStream_t s);
// Blockwise FP8 variant: block = 1 (1 x 128 activation blocks, scale[kb][rows])
// or 128 (128 x 128 weight blocks, scale[row block][kb]).
mx_status launch_quantize_blockwise(const void* x, int64_t rows, int64_t cols, int64_t ldx, int block, void* data,
                                    float* scale, cudaStream_t s);

// --- GEMM ------------------------------------------------------------------
enum GemmKind { GEMM_DENSE = 0, GEMM_GROUPED_M = 1, GEMM_GROUPED_K = 2 };

// The epilogue of mx_gemm_epilogue; null pointers: not there.
struct GemmEpilogue {
  const void* bias;      // N entries
  const void* residual;  // BF16 [M, N]
  void* preact;          // BF16 [M, N], written
  int64_t ld_residual;
  int64_t ld_preact;
  int32_t bias_f32;
  int32_t act;           // mx_act
};

struct GemmLaunch {
  GemmKind kind;
  const void* a_data;
  const void* a_scale;
  int64_t a_ld;
  const void* b_data;
  const void* b_scale;
  int64_t b_ld;
  int64_t M;        // rows of C (per group for GROUPED_K)
  int64_t N;        // columns of C
  int64_t K;        // contraction length (capacity for GROUPED_K)
  int64_t b_rows_total;  // rows of the 2-D view of b (E*N for GROUPED_M, else N)
  void* c;
  int64_t ldc;
  const int64_t* offsets;
  int n_groups;
  int* dev_status;
  bool swiglu = false;  // rows-ragged only: C = SwiGLU(A . B^T), gate = B rows [0, N/2), up = [N/2, N)
  // Blockwise FP8 variant (dense): FP32 multipliers of A's 1 x 128 blocks
  // ([K/128][M]) and B's 128 x 128 blocks ([ceil(N/128)][K/128]); a_scale /
  // b_scale unused.
  const float* bw_a_scale = nullptr;
  const float* bw_b_scale = nullptr;
  // The caller's workspace for the dense split tail; without one (or with
  // too small a one) the GEMM runs whole tiles only.
  void* ws = nullptr;
  size_t ws_bytes = 0;
  // Current-scaling recipe: a_scale / b_scale are FP32 tensor scales (b: one
  // per expert for rows-ragged grouped GEMMs) applied in the epilogue.
  bool tensor_scaled = false;
  // Rows-ragged SwiGLU only: instead of the BF16 output, its MX copies as
  // mx_quantize (both copies, per-expert column segments) would write them from
  // that output: row copy [M, N/2] + scales, column copy [N/2, q_cap] + scales.
  void* q_row_data = nullptr;
  void* q_row_scale = nullptr;
  void* q_col_data = nullptr;
  void* q_col_scale = nullptr;
  int64_t q_cap = 0;
  // Dense, block-scaled only: C = act(A . B^T + bias) + residual (whole tiles,
  // no split tail).
  bool has_epi = false;
  GemmEpilogue epi = {};
  // Dense, block-scaled only (mx_gemm_gated): b is the gate's operand, this one the
  // up projection's; N counts both (2F), C = act(A . B^T) * (A . up^T) has F
  // columns; epi.preact (with ld_preact) and epi.act are read.
  const void* up_data = nullptr;
  const void* up_scale = nullptr;
  int64_t up_ld = 0;
};
mx_status launch_gemm(const GemmLaunch& g, cudaStream_t s);
// The gated product of few tiles (up_data set): whether it takes this launch, and it.
bool gated_few_applies(const GemmLaunch& g);
mx_status launch_gated_few(const GemmLaunch& g, cudaStream_t s);
// An operand's map: box 128 K x box_rows, 128-byte swizzle, zeros outside.
mx_status make_operand_map(CUtensorMap* map, const void* base, int64_t rows, int64_t k, int64_t ld, int box_rows);
// Bytes of workspace the dense GEMM L would use for its split tail (0: none).
size_t gemm_workspace_bytes(const GemmLaunch& L);
// Device address and size of the library's static scratch array on the
// current device (looked up on the first call per device).
mx_status static_workspace(void** ptr, size_t* bytes);
// Up to MX_MAX_GEMM_MULTI independent dense GEMMs; one launch of the pair
// kernel when they fill the GPU together, else one launch each.
mx_status launch_gemm_multi(const GemmLaunch* Ls, int n, cudaStream_t s);

// --- operators around the products -----------------------------------------
mx_status launch_adamw(const mx_adamw_tensor* tensors, int n, int bits, const mx_adamw_hyper& hy,
                       const float* grad_scale, int* dev_status, cudaStream_t s);

// The epilogue alone, on a product that is zero (empty contraction).
mx_status launch_epilogue_only(const GemmEpilogue& e, int64_t M, int64_t N, void* c, int64_t ldc, cudaStream_t s);

struct EpilogueBackwardLaunch {
  const void* dy;
  int64_t lddy;
  const void* z;  // unused with MX_ACT_NONE
  int64_t ldz;
  int64_t rows, cols;
  int act;
  void* dz;  // may be null
  int64_t lddz;
  float* dbias;  // may be null
  void* ws;
};
mx_status launch_epilogue_backward(const EpilogueBackwardLaunch& L, cudaStream_t s);
size_t epilogue_backward_workspace(int64_t rows, int64_t cols);

struct RouterLaunch {
  const void* logits;
  int64_t ld;
  int dtype;
  const uint8_t* mask;  // may be null
  int64_t tokens, tokens_per_seq;
  int experts, top_k, normalize;
  float coef;             // forward
  int32_t* indices;       // written (forward), read (backward)
  float* weights;         // forward outputs ...
  int64_t* counts;
  int64_t* offsets;
  float* load;            // written (forward), read (backward)
  float* loss;
  void* ws;
  const float* dweights;  // backward inputs (may be null) and output
  const float* dloss;
  void* dlogits;
  int64_t lddx;
};
mx_status launch_router_forward(const RouterLaunch& L, cudaStream_t s);
mx_status launch_router_backward(const RouterLaunch& L, cudaStream_t s);
size_t router_workspace(int64_t tokens, int64_t tokens_per_seq, int experts);
// Whether the launch's CTAs can be counted.
bool router_fits(int64_t tokens, int64_t tokens_per_seq, int experts);

struct NormLaunch {
  const void* x;
  int64_t ldx;
  const void* dy;  // backward
  int64_t lddy;
  const void* weight;  // null: 1
  const void* bias;    // null: 0
  int param_dtype;
  int64_t rows, cols;
  int dtype;
  int center;
  float eps;
  void* out;  // y or dx
  int64_t ldo;
  float* mean;
  float* rstd;
  float* dweight;  // backward, may be null
  float* dbias;
  void* ws;
  int* dev_status;
  // The self test of the stages' waits: their limit (0: the library's), and the
  // bytes that each waits for in vain.
  uint64_t timeout_ns;
  uint32_t withheld;
};
mx_status launch_norm_forward(const NormLaunch& L, cudaStream_t s);
mx_status launch_norm_backward(const NormLaunch& L, cudaStream_t s);
size_t norm_backward_workspace(int64_t rows, int64_t cols);
// Tensor map over a [rows, cols] matrix (pitch ld elements) in boxes of 32 rows of
// 128 bytes, 128-byte swizzle: BF16 boxes of 64 columns, FP32 ones of 32. box_rows:
// fewer in the self test, whose stages wait for the rest in vain.
mx_status make_unit_map(CUtensorMap* map, bool f32, const void* base, int64_t cols, int64_t rows, int64_t ld,
                        int box_rows = 32);

struct AddNormLaunch {
  bool backward;
  bool stream_f32;      // residual and sum (backward: sum, dsum and dx) are FP32
  const void* first;    // x; backward: dy (BF16)
  int64_t ld_first;
  const void* second;   // residual (may be null); backward: sum
  int64_t ld_second;
  const void* third;    // backward: dsum (may be null)
  int64_t ld_third;
  const void* weight;   // may be null
  int param_dtype;
  int64_t rows, cols;
  float eps;
  void* out;            // sum (may be null); backward: dx
  int64_t ld_out;
  void* y;              // forward, may be null
  int64_t ldy;
  float* rstd;          // written (may be null); backward: read
  void* row_data;       // null: no row copy
  void* row_scale;
  void* col_data;       // null: no column copy
  void* col_scale;
  float* dweight;       // backward, may be null
  void* ws;
  int* dev_status;
};
mx_status launch_add_norm(const AddNormLaunch& L, cudaStream_t s);
size_t add_norm_backward_workspace(int64_t rows, int64_t cols);

struct GatedLaunch {
  const void* dh;       // backward (BF16 [rows, F]); null: forward
  int64_t lddh;
  const void* gate_up;  // BF16 [rows, 2F]
  int64_t ld;
  int64_t rows, f;
  int act;
  void* row_data;       // null: no row copy
  void* row_scale;
  void* col_data;       // null: no column copy
  void* col_scale;
  const int64_t* offsets;  // null: dense
  int n_groups;
  int64_t col_pitch;    // rows (dense) or the capacity
  int* dev_status;
};
mx_status launch_gated(const GatedLaunch& L, cudaStream_t s);

// Sums over p < parts of partial[p][c], added in a fixed order: columns [0, n0)
// to out0, [n0, n0 + n1) to out1 (null: not wanted). hold_next: the next kernel on the
// stream starts behind it, not beside it.
mx_status launch_column_reduce(const float* partial, int parts, int64_t n0, int64_t n1, float* out0, float* out1,
                               cudaStream_t s, bool hold_next = false);

}  // namespace mx
