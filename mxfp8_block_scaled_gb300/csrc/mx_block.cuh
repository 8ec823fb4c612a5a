// A warp's unit of 32 rows x 64 columns: FP32 values in registers -> MX row and
// column copies (the codec and layouts of mx_codec.cuh), for the kernels that
// quantise what they compute. Blocks are formed from the FP32 values: amax, scale
// and elements, with one rounding, to E4M3.
//
// Lane 8 g + q holds rows 8 g .. 8 g + 7 and columns 8 q .. 8 q + 7, so that
// - eight lanes read a whole 128-byte row of a shared-memory box, without bank
//   conflicts whatever the row;
// - a row's block is four lanes' and a column's four too, 8 rows x 8 columns of a
//   lane: in each direction the four lanes fold their amaxes (two to a register)
//   until each has two blocks' whole ones (3 shuffles), and hand the two scales
//   round (3 more);
// - a lane's codes of a row are an 8-byte store, eight lanes 64 bytes of the row;
//   its codes of a column are one too, four lanes a 32-byte sector.
// An amax is kept as the high half of its FP32 pattern: the exponent decides the
// scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mx_codec.cuh"
#include "mx_ptx.cuh"

namespace mx {

constexpr int kUnitRows = 32;
constexpr int kUnitCols = 64;

__device__ __forceinline__ void st_shared_v2(void* p, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(smem_u32(p)), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_shared_u8(void* p, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}

// Where a matrix's MX copies go.
struct CopyOut {
  uint8_t* row_data;
  uint8_t* row_scale;
  uint8_t* col_data;
  uint8_t* col_scale;
  int64_t row_pitch;  // bytes: the matrix's columns
  int64_t row_ka;     // scale-column atoms of the row copy
  int64_t col_pitch;  // bytes: the column copy's contraction length
  int64_t col_ka;     // scale-column atoms of the column copy
};

// Largest magnitude of three; NaN if one is NaN.
__device__ __forceinline__ float amax3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// Four values -> four E4M3 codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t unit_cvt(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

// The E8M0 codes (two 16-bit fields) of two amaxes' high halves: floor(log2) - 8 +
// 127, at least 0; 247 for Inf and NaN, which the caller replaces.
__device__ __forceinline__ uint32_t unit_codes(uint32_t amax2) {
  return __vmaxu2((amax2 >> 7) & 0x00FF00FFu, 0x00080008u) - 0x00080008u;
}

// Folds the amaxes of a lane's eight rows (or columns), two to a register, over the
// four lanes that share their blocks (lane bits `a` and `b` of it): the lane ends
// with pair 2 b + a whole.
__device__ __forceinline__ uint32_t unit_fold(const uint32_t (&p)[4], bool a, bool b, int xa, int xb) {
  uint32_t s0 = __vmaxu2(b ? p[2] : p[0], __shfl_xor_sync(0xFFFFFFFFu, b ? p[0] : p[2], xb));
  uint32_t s1 = __vmaxu2(b ? p[3] : p[1], __shfl_xor_sync(0xFFFFFFFFu, b ? p[1] : p[3], xb));
  return __vmaxu2(a ? s1 : s0, __shfl_xor_sync(0xFFFFFFFFu, a ? s0 : s1, xa));
}

// The other way: each lane's pair to all four, in order.
__device__ __forceinline__ void unit_gather(uint32_t mine, bool a, bool b, int xa, int xb, uint32_t (&out)[4]) {
  const uint32_t t = __shfl_xor_sync(0xFFFFFFFFu, mine, xa);
  const uint32_t e0 = a ? t : mine, e1 = a ? mine : t;
  const uint32_t f0 = __shfl_xor_sync(0xFFFFFFFFu, e0, xb), f1 = __shfl_xor_sync(0xFFFFFFFFu, e1, xb);
  out[0] = b ? f0 : e0;
  out[1] = b ? f1 : e1;
  out[2] = b ? e0 : f0;
  out[3] = b ? e1 : f1;
}

// scale_offset for rows and blocks below 2^31.
__device__ __forceinline__ int64_t unit_scale_offset(uint32_t r, uint32_t kb, int64_t ka) {
  return ((static_cast<int64_t>(r >> 7) * ka + (kb >> 2)) << 9) + (((r & 31) << 4) + (((r >> 5) & 3) << 2) + (kb & 3));
}

// Two fields of 16 bits, each all ones where the amax there is Inf or NaN.
__device__ __forceinline__ uint32_t unit_bad(uint32_t amax2) {
  return ((amax2 & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((amax2 & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// Whether some lane of the warp has one (code 247).
__device__ __forceinline__ bool unit_any_bad(uint32_t codes) {
  return __any_sync(0xFFFFFFFFu, ((codes + 0x00090009u) & 0x01000100u) != 0u);
}

// One unit to its copies. v[i][j]: row 8 g + i, columns 8 q + 2 j and + 1.
//   row0, c0  the unit's first row and column in the matrix; c_end the matrix's
//             columns (a multiple of 32; values past it are not read)
//   rows      how many of its rows exist: others have no row copy. The column
//             copy takes all 32 (the caller has zeroed what does not exist).
//   kpos      position of its first row along the column copy's contraction.
//   staged    not null: the column copy's codes and scales of panel `panel` (of four)
//             go to this tile in shared memory instead, for store_columns.
// A block with Inf or NaN takes scale 0xFF and codes 0x7F with the sign that the
// element's conversion has.
template <bool kRow, bool kCol, bool kStaged = false>
__device__ __forceinline__ void store_unit(const float2 (&v)[8][4], const CopyOut& o, int lane, int64_t row0, int rows,
                                           int64_t c0, int64_t c_end, int64_t kpos, uint8_t* staged = nullptr,
                                           int panel = 0) {
  const int q = lane & 7, g = lane >> 3;
  const int64_t c = c0 + 8 * q;
  const bool in = c < c_end;  // blocks are whole: so are a lane's columns
  if constexpr (kRow) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float m[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2(&r)[4] = v[i + k];
        m[k] = amax3(amax3(r[0].x, r[0].y, r[1].x), amax3(r[1].y, r[2].x, r[2].y), amax3(r[3].x, r[3].y, 0.0f));
      }
      p[i >> 1] = high_halves(m[0], m[1]);
    }
    const bool a = (q & 1) != 0, b = (q & 2) != 0;
    const uint32_t amax = unit_fold(p, a, b, 1, 2);  // rows 8 g + 2 (q % 4) and + 1, this block
    uint32_t codes = unit_codes(amax);
    uint32_t inv[4];  // 2^-X of the eight rows, as BF16
    unit_gather((0x00FE00FEu - codes) << 7, a, b, 1, 2, inv);
    uint32_t bads[4] = {0u, 0u, 0u, 0u};
    const bool any_bad = unit_any_bad(codes);
    if (any_bad) {
      const uint32_t bad = unit_bad(amax);
      codes |= bad & 0x00FF00FFu;
      unit_gather(bad, a, b, 1, 2, bads);
    }
    uint8_t* dst = o.row_data + (row0 + 8 * g) * o.row_pitch + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = (i & 1) ? hi_f(inv[i >> 1]) : lo_f(inv[i >> 1]);
      const float2 s = make_float2(f, f);
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 x = __fmul2_rn(v[i][2 * j], s), y = __fmul2_rn(v[i][2 * j + 1], s);
        w[j] = unit_cvt(x.x, x.y, y.x, y.y);
      }
      if (any_bad) {
        const uint32_t fill = ((i & 1) ? bads[i >> 1] >> 16 : bads[i >> 1] & 0xFFFFu) ? 0x7F7F7F7Fu : 0u;
        w[0] |= fill;
        w[1] |= fill;
      }
      if (in && 8 * g + i < rows) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      dst += o.row_pitch;
    }
    // The lanes of the first block write row 8 g + 2 (q % 4), both blocks' scales,
    // those of the second the row behind it.
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, codes, 4);
    const bool second = (q & 4) != 0;
    const uint32_t lo = second ? other >> 16 : codes, hi = second ? codes >> 16 : other;
    const int r = 8 * g + 2 * (q & 3) + (second ? 1 : 0);
    if (r < rows) {
      const uint32_t kb = static_cast<uint32_t>(c0) >> 5;
      uint8_t* at = o.row_scale + unit_scale_offset(static_cast<uint32_t>(row0) + r, kb, o.row_ka);
      if (c0 + 32 < c_end && (kb & 1) == 0) {
        *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>((lo & 0xFFu) | ((hi & 0xFFu) << 8));
      } else {
        *at = static_cast<uint8_t>(lo);
        if (c0 + 32 < c_end)
          o.row_scale[unit_scale_offset(static_cast<uint32_t>(row0) + r, kb + 1, o.row_ka)] = static_cast<uint8_t>(hi);
      }
    }
  }
  if constexpr (kCol) {
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = amax3(amax3(v[0][j].x, v[1][j].x, v[2][j].x), amax3(v[3][j].x, v[4][j].x, v[5][j].x),
                            amax3(v[6][j].x, v[7][j].x, 0.0f));
      const float y = amax3(amax3(v[0][j].y, v[1][j].y, v[2][j].y), amax3(v[3][j].y, v[4][j].y, v[5][j].y),
                            amax3(v[6][j].y, v[7][j].y, 0.0f));
      p[j] = high_halves(x, y);
    }
    const bool a = (g & 1) != 0, b = (g & 2) != 0;
    const uint32_t amax = unit_fold(p, a, b, 8, 16);  // columns 8 q + 2 g and + 1
    uint32_t codes = unit_codes(amax);
    uint32_t inv[4];
    unit_gather((0x00FE00FEu - codes) << 7, a, b, 8, 16, inv);
    uint32_t bads[4] = {0u, 0u, 0u, 0u};
    const bool any_bad = unit_any_bad(codes);
    if (any_bad) {
      const uint32_t bad = unit_bad(amax);
      codes |= bad & 0x00FF00FFu;
      unit_gather(bad, a, b, 8, 16, bads);
    }
    uint8_t* dst = kStaged ? staged + q * 1024 + (((panel * 2 + (g >> 1)) ^ q) << 4) + (g & 1) * 8
                           : o.col_data + c * o.col_pitch + kpos + 8 * g;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 s = make_float2(lo_f(inv[j]), hi_f(inv[j]));
      uint32_t w0[2], w1[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 x0 = __fmul2_rn(v[4 * k][j], s), x1 = __fmul2_rn(v[4 * k + 1][j], s),
                     x2 = __fmul2_rn(v[4 * k + 2][j], s), x3 = __fmul2_rn(v[4 * k + 3][j], s);
        w0[k] = unit_cvt(x0.x, x1.x, x2.x, x3.x);
        w1[k] = unit_cvt(x0.y, x1.y, x2.y, x3.y);
      }
      if (any_bad) {
        const uint32_t f0 = (bads[j] & 0xFFFFu) ? 0x7F7F7F7Fu : 0u, f1 = (bads[j] >> 16) ? 0x7F7F7F7Fu : 0u;
        w0[0] |= f0;
        w0[1] |= f0;
        w1[0] |= f1;
        w1[1] |= f1;
      }
      if constexpr (kStaged) {
        st_shared_v2(dst + 256 * j, w0[0], w0[1]);
        st_shared_v2(dst + 256 * j + 128, w1[0], w1[1]);
      } else {
        if (in) {
          *reinterpret_cast<uint2*>(dst) = make_uint2(w0[0], w0[1]);
          *reinterpret_cast<uint2*>(dst + o.col_pitch) = make_uint2(w1[0], w1[1]);
        }
        dst += 2 * o.col_pitch;
      }
    }
    if constexpr (kStaged) {
      uint8_t* at = staged + kUnitCols * 128 + (8 * q + 2 * g) * 4 + panel;
      st_shared_u8(at, codes);
      st_shared_u8(at + 4, codes >> 16);
    } else if (in) {
      // An even column and the one behind it: 16 bytes further on.
      uint8_t* at = o.col_scale + unit_scale_offset(static_cast<uint32_t>(c) + 2 * g, static_cast<uint32_t>(kpos) >> 5, o.col_ka);
      at[0] = static_cast<uint8_t>(codes);
      at[16] = static_cast<uint8_t>(codes >> 16);
    }
  }
}

// A tile of four panels' column copies that store_unit staged: 64 columns of 128
// codes (16-byte chunk n of column c at n ^ (c / 8)), then their four scales each.
// Written whole: 128 bytes a column where 32 at a time, from warps that are not at
// the same place, left the lines to L2's fortune (dense backward, 8192 x 10944: 147
// to 190 us with the order of the tiles). Warp w of four writes columns 16 w .. 16 w +
// 15; k_end: the copy's contraction length where the last tile may pass it.
constexpr int kStagedBytes = kUnitCols * 128 + kUnitCols * 4;

__device__ __forceinline__ void store_columns(const uint8_t* staged, const CopyOut& o, int warp, int lane, int64_t c0,
                                              int64_t c_end, int64_t kpos, int64_t k_end) {
  const int chunk = lane & 7;
  const int col0 = 16 * warp + (lane >> 3);
  uint8_t* dst = o.col_data + (c0 + col0) * o.col_pitch + kpos + chunk * 16;
  const bool in = kpos + chunk * 16 < k_end;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int col = col0 + 4 * it;
    const uint4 w = ld_shared_v4(staged + col * 128 + ((chunk ^ (col >> 3)) << 4));
    if (in && c0 + col < c_end) *reinterpret_cast<uint4*>(dst) = w;
    dst += 4 * o.col_pitch;
  }
  const int c = 16 * warp + lane;
  if (lane < 16 && c0 + c < c_end)
    *reinterpret_cast<uint32_t*>(o.col_scale + unit_scale_offset(static_cast<uint32_t>(c0) + c, static_cast<uint32_t>(kpos) >> 5,
                                                                 o.col_ka)) =
        *reinterpret_cast<const uint32_t*>(staged + kUnitCols * 128 + c * 4);
}

// Zeros in the scale buffer of a copy (rows x kb blocks, ka atoms wide) that belong
// to no block: blocks up to a multiple of four, rows up to a multiple of 128.
// Threads `id` of `n`.
__device__ __forceinline__ void zero_scale_padding(uint8_t* scale, int64_t rows, int64_t kb, int64_t ka, int64_t id,
                                                   int64_t n) {
  const int64_t atoms = (kb + 3) >> 2, padded = (rows + 127) & ~int64_t{127};
  if (kb & 3)
    for (int64_t r = id; r < rows; r += n)
      for (int64_t b = kb; b < 4 * atoms; ++b) scale[scale_offset(r, b, ka)] = 0;
  const int64_t left = (padded - rows) * atoms;
  for (int64_t i = id; i < left; i += n)
    *reinterpret_cast<uint32_t*>(scale + scale_offset(rows + i / atoms, 4 * (i % atoms), ka)) = 0u;
}

// A lane's 8 columns of row r (of 32) of a unit in shared memory: a [32][64] BF16
// box or two [32][32] FP32 boxes, 128-byte rows, 16-byte chunk n of row r at
// n ^ (r % 8). The second FP32 box starts a row further on (kF32Box): its chunks
// are swizzled by r + 1, so that the eight lanes of a row, four in each box, meet
// different banks.
constexpr int kF32Box = 4096 + 128;
__host__ __device__ constexpr uint32_t unit_box_bytes(bool f32) { return f32 ? 9216 : 4096; }  // with the row between the boxes, to 1024

__device__ __forceinline__ void unit_row_bf16(const uint8_t* box, int r, int q, float2 (&out)[4]) {
  const uint4 w = ld_shared_v4(box + r * 128 + ((q ^ (r & 7)) << 4));
  out[0] = make_float2(lo_f(w.x), hi_f(w.x));
  out[1] = make_float2(lo_f(w.y), hi_f(w.y));
  out[2] = make_float2(lo_f(w.z), hi_f(w.z));
  out[3] = make_float2(lo_f(w.w), hi_f(w.w));
}

__device__ __forceinline__ void unit_row_f32(const uint8_t* boxes, int r, int q, float2 (&out)[4]) {
  const int second = q >> 2;
  const uint8_t* box = boxes + second * kF32Box;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 w = ld_shared_v4(box + r * 128 + (((2 * (q & 3) + h) ^ ((r + second) & 7)) << 4));
    out[2 * h] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    out[2 * h + 1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}

template <bool kF32>
__device__ __forceinline__ void unit_row(const uint8_t* box, int r, int q, float2 (&out)[4]) {
  if constexpr (kF32) unit_row_f32(box, r, q, out);
  else unit_row_bf16(box, r, q, out);
}

// A lane's 8 columns of a row to memory, rounded to the element type.
template <bool kF32>
__device__ __forceinline__ void store_row(void* base, int64_t at, const float2 (&v)[4]) {
  if constexpr (kF32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) d[h] = make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[j].x, v[j].y);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A lane's 8 columns of a row from memory.
template <bool kF32>
__device__ __forceinline__ void load_row(const void* base, int64_t at, float2 (&v)[4]) {
  if constexpr (kF32) {
    const float4* d = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 t = d[h];
      v[2 * h] = make_float2(t.x, t.y);
      v[2 * h + 1] = make_float2(t.z, t.w);
    }
  } else {
    const uint4 t = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    v[0] = make_float2(lo_f(t.x), hi_f(t.x));
    v[1] = make_float2(lo_f(t.y), hi_f(t.y));
    v[2] = make_float2(lo_f(t.z), hi_f(t.z));
    v[3] = make_float2(lo_f(t.w), hi_f(t.w));
  }
}

// Sum over a unit's columns of eight row sums a lane: lane l gets row l's.
__device__ __forceinline__ float fold_rows(const float (&s)[8], int lane) {
  const bool a = (lane & 1) != 0, b = (lane & 2) != 0, d = (lane & 4) != 0;
  float t[4], u[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = (d ? s[i + 4] : s[i]) + __shfl_xor_sync(0xFFFFFFFFu, d ? s[i] : s[i + 4], 4);
#pragma unroll
  for (int i = 0; i < 2; ++i) u[i] = (b ? t[i + 2] : t[i]) + __shfl_xor_sync(0xFFFFFFFFu, b ? t[i] : t[i + 2], 2);
  return (a ? u[1] : u[0]) + __shfl_xor_sync(0xFFFFFFFFu, a ? u[0] : u[1], 1);
}

}  // namespace mx
