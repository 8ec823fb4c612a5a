// A warp's unit of 32 rows x 64 columns: FP32 values in registers -> MX row and
// column copies (the codec and layouts of mx_codec.cuh), for the kernels that
// quantise what they compute. Blocks are formed from the FP32 values: amax, scale
// and elements, with one rounding, to E4M3.
//
// Lane 4 g + q holds rows 4 g .. 4 g + 3 and columns 16 q .. 16 q + 15, so that
// - a row's block is two neighbouring lanes' (one shuffle for the amax, of two rows
//   a register), and a lane's codes of a row are one 16-byte store (a quarter of
//   the warp's 64 bytes of that row);
// - a column's block is eight lanes' (columns split among them step by step: 7
//   shuffles for 64 columns, 4 more to hand the scales back), and its 32 codes
//   leave as eight 4-byte pieces of one 32-byte sector.
// An amax is kept as the high half of its FP32 pattern (the exponent decides the
// scale), two to a register. About 240 instructions for a lane's 64 values with
// both copies, a tenth of the issue slots that HBM leaves at 8 bytes a value.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mx_codec.cuh"
#include "mx_ptx.cuh"

namespace mx {

constexpr int kUnitRows = 32;
constexpr int kUnitCols = 64;

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

// 2^-X of scale code number i of four packed ones (255 as 0: its codes are replaced).
__device__ __forceinline__ float unit_inv(uint32_t minus, int i) {
  return __uint_as_float(__byte_perm(minus, 0u, i == 0 ? 0x0444 : i == 1 ? 0x1444 : i == 2 ? 0x2444 : 0x3444) >> 1);
}

// 254 - code in each byte, 254 for the code 255.
__device__ __forceinline__ uint32_t minus_codes(uint32_t codes) {
  const uint32_t nan = __vcmpeq4(codes, 0xFFFFFFFFu);
  return 0xFEFEFEFEu - (codes & ~nan);
}

__device__ __forceinline__ uint32_t nan_code(float v) { return 0x7Fu | ((__float_as_uint(v) >> 24) & 0x80u); }

// One unit to its copies. v[i][j]: row 4 g + i, columns 16 q + 2 j and + 1.
//   row0, c0  the unit's first row and column in the matrix; c_end the matrix's
//             columns (a multiple of 32; values past it are not read)
//   rows      how many of its rows exist: others have no row copy. The column
//             copy takes all 32 (the caller has zeroed what does not exist).
//   kpos      position of its first row along the column copy's contraction.
template <bool kRow, bool kCol>
__device__ __forceinline__ void store_unit(const float2 (&v)[4][8], const CopyOut& o, int lane, int64_t row0, int rows,
                                           int64_t c0, int64_t c_end, int64_t kpos) {
  const int q = lane & 3, g = lane >> 2;
  const int64_t c = c0 + 16 * q;
  const bool in = c < c_end;  // blocks are whole: so are a lane's 16 columns
  if constexpr (kRow) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = amax3(v[i][0].x, v[i][0].y, v[i][1].x);
      m[i] = amax3(m[i], v[i][1].y, v[i][2].x);
#pragma unroll
      for (int j = 2; j < 7; ++j) m[i] = amax3(m[i], v[i][j].y, v[i][j + 1].x);
      m[i] = amax3(m[i], v[i][7].y, 0.0f);
    }
    uint32_t p0 = high_halves(m[0], m[1]), p1 = high_halves(m[2], m[3]);
    p0 = __vmaxu2(p0, __shfl_xor_sync(0xFFFFFFFFu, p0, 1));
    p1 = __vmaxu2(p1, __shfl_xor_sync(0xFFFFFFFFu, p1, 1));
    const uint32_t codes = scale_code(p0 & 0xFFFFu) | (scale_code(p0 >> 16) << 8) | (scale_code(p1 & 0xFFFFu) << 16) |
                           (scale_code(p1 >> 16) << 24);
    const uint32_t minus = minus_codes(codes);
    const uint32_t nans = __vcmpeq4(codes, 0xFFFFFFFFu);
    const bool any_nan = __any_sync(0xFFFFFFFFu, nans != 0u);
    uint8_t* dst = o.row_data + (row0 + 4 * g) * o.row_pitch + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float inv = unit_inv(minus, i);
      const float2 s = make_float2(inv, inv);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = __fmul2_rn(v[i][2 * j], s), b = __fmul2_rn(v[i][2 * j + 1], s);
        w[j] = cvt_pair(a.x, a.y) | (cvt_pair(b.x, b.y) << 16);
      }
      if (any_nan && ((nans >> (8 * i)) & 1u)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = nan_code(v[i][2 * j].x) | (nan_code(v[i][2 * j].y) << 8) | (nan_code(v[i][2 * j + 1].x) << 16) |
                 (nan_code(v[i][2 * j + 1].y) << 24);
      }
      if (in && 4 * g + i < rows) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      dst += o.row_pitch;
    }
    // Lane l writes both blocks' scales of row l.
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, codes, 2);
    const uint32_t lo = ((q & 2) ? other : codes) >> (8 * q), hi = ((q & 2) ? codes : other) >> (8 * q);
    if (lane < rows) {
      const int64_t kb = c0 >> 5, r = row0 + lane;
      if (c0 + 32 < c_end && (kb & 1) == 0) {
        *reinterpret_cast<uint16_t*>(o.row_scale + scale_offset(r, kb, o.row_ka)) =
            static_cast<uint16_t>((lo & 0xFFu) | ((hi & 0xFFu) << 8));
      } else {
        o.row_scale[scale_offset(r, kb, o.row_ka)] = static_cast<uint8_t>(lo);
        if (c0 + 32 < c_end) o.row_scale[scale_offset(r, kb + 1, o.row_ka)] = static_cast<uint8_t>(hi);
      }
    }
  }
  if constexpr (kCol) {
    uint32_t p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = amax3(amax3(v[0][j].x, v[1][j].x, v[2][j].x), v[3][j].x, 0.0f);
      const float y = amax3(amax3(v[0][j].y, v[1][j].y, v[2][j].y), v[3][j].y, 0.0f);
      p[j] = high_halves(x, y);
    }
    // Lane 4 g + q ends with pair g: columns 16 q + 2 g and + 1.
    const bool b2 = (g & 4) != 0, b1 = (g & 2) != 0, b0 = (g & 1) != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t t = __shfl_xor_sync(0xFFFFFFFFu, b2 ? p[j] : p[j + 4], 16);
      p[j] = __vmaxu2(b2 ? p[j + 4] : p[j], t);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t t = __shfl_xor_sync(0xFFFFFFFFu, b1 ? p[j] : p[j + 2], 8);
      p[j] = __vmaxu2(b1 ? p[j + 2] : p[j], t);
    }
    {
      const uint32_t t = __shfl_xor_sync(0xFFFFFFFFu, b0 ? p[0] : p[1], 4);
      p[0] = __vmaxu2(b0 ? p[1] : p[0], t);
    }
    const uint32_t mine = scale_code(p[0] & 0xFFFFu) | (scale_code(p[0] >> 16) << 8);
    // The sixteen codes of the lane's columns, four to a word, from the eight lanes.
    uint32_t k0, k1, k2, k3;
    {
      const uint32_t t = __shfl_xor_sync(0xFFFFFFFFu, mine, 4);
      const uint32_t four = b0 ? __byte_perm(t, mine, 0x5410) : __byte_perm(mine, t, 0x5410);
      const uint32_t f2 = __shfl_xor_sync(0xFFFFFFFFu, four, 8);
      const uint32_t e0 = b1 ? f2 : four, e1 = b1 ? four : f2;
      const uint32_t s0 = __shfl_xor_sync(0xFFFFFFFFu, e0, 16), s1 = __shfl_xor_sync(0xFFFFFFFFu, e1, 16);
      k0 = b2 ? s0 : e0;
      k1 = b2 ? s1 : e1;
      k2 = b2 ? e0 : s0;
      k3 = b2 ? e1 : s1;
    }
    const bool any_nan = __any_sync(0xFFFFFFFFu, __vcmpeq4(k0, ~0u) | __vcmpeq4(k1, ~0u) | __vcmpeq4(k2, ~0u) |
                                                     __vcmpeq4(k3, ~0u));
    uint8_t* dst = o.col_data + c * o.col_pitch + kpos + 4 * g;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t k = j < 2 ? k0 : j < 4 ? k1 : j < 6 ? k2 : k3;
      const uint32_t minus = minus_codes(k);
      const float2 s = make_float2(unit_inv(minus, (2 * j) & 3), unit_inv(minus, (2 * j + 1) & 3));
      const float2 a = __fmul2_rn(v[0][j], s), b = __fmul2_rn(v[1][j], s), d = __fmul2_rn(v[2][j], s),
                   e = __fmul2_rn(v[3][j], s);
      uint32_t w0 = cvt_pair(a.x, b.x) | (cvt_pair(d.x, e.x) << 16);
      uint32_t w1 = cvt_pair(a.y, b.y) | (cvt_pair(d.y, e.y) << 16);
      if (any_nan) {
        if (((k >> (8 * ((2 * j) & 3))) & 0xFFu) == 0xFFu)
          w0 = nan_code(v[0][j].x) | (nan_code(v[1][j].x) << 8) | (nan_code(v[2][j].x) << 16) | (nan_code(v[3][j].x) << 24);
        if (((k >> (8 * ((2 * j + 1) & 3))) & 0xFFu) == 0xFFu)
          w1 = nan_code(v[0][j].y) | (nan_code(v[1][j].y) << 8) | (nan_code(v[2][j].y) << 16) | (nan_code(v[3][j].y) << 24);
      }
      if (in) {
        *reinterpret_cast<uint32_t*>(dst) = w0;
        *reinterpret_cast<uint32_t*>(dst + o.col_pitch) = w1;
      }
      dst += 2 * o.col_pitch;
    }
    if (in) {
      o.col_scale[scale_offset(c + 2 * g, kpos >> 5, o.col_ka)] = static_cast<uint8_t>(mine);
      o.col_scale[scale_offset(c + 2 * g + 1, kpos >> 5, o.col_ka)] = static_cast<uint8_t>(mine >> 8);
    }
  }
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

// A lane's 16 columns of row r (of 32) of a unit in shared memory: a [32][64] BF16
// box or two [32][32] FP32 boxes, 128-byte rows, 16-byte chunk n of row r at
// n ^ (r % 8).
__device__ __forceinline__ void unit_row_bf16(const uint8_t* box, int r, int q, float2 (&out)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 w = ld_shared_v4(box + r * 128 + (((2 * q + h) ^ (r & 7)) << 4));
    out[4 * h + 0] = make_float2(lo_f(w.x), hi_f(w.x));
    out[4 * h + 1] = make_float2(lo_f(w.y), hi_f(w.y));
    out[4 * h + 2] = make_float2(lo_f(w.z), hi_f(w.z));
    out[4 * h + 3] = make_float2(lo_f(w.w), hi_f(w.w));
  }
}

__device__ __forceinline__ void unit_row_f32(const uint8_t* boxes, int r, int q, float2 (&out)[8]) {
  const uint8_t* box = boxes + (q >> 1) * 4096;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint4 w = ld_shared_v4(box + r * 128 + (((4 * (q & 1) + h) ^ (r & 7)) << 4));
    out[2 * h] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    out[2 * h + 1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}

template <bool kF32>
__device__ __forceinline__ void unit_row(const uint8_t* box, int r, int q, float2 (&out)[8]) {
  if constexpr (kF32) unit_row_f32(box, r, q, out);
  else unit_row_bf16(box, r, q, out);
}

// A lane's 16 columns of a row to memory, rounded to the element type.
template <bool kF32>
__device__ __forceinline__ void store_row(void* base, int64_t at, const float2 (&v)[8]) {
  if constexpr (kF32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
#pragma unroll
    for (int h = 0; h < 4; ++h) d[h] = make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y);
  } else {
    uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[4 * h + j].x, v[4 * h + j].y);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      d[h] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// A lane's 16 columns of a row from memory.
template <bool kF32>
__device__ __forceinline__ void load_row(const void* base, int64_t at, float2 (&v)[8]) {
  if constexpr (kF32) {
    const float4* d = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float4 t = d[h];
      v[2 * h] = make_float2(t.x, t.y);
      v[2 * h + 1] = make_float2(t.z, t.w);
    }
  } else {
    const uint4* d = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 t = d[h];
      v[4 * h] = make_float2(lo_f(t.x), hi_f(t.x));
      v[4 * h + 1] = make_float2(lo_f(t.y), hi_f(t.y));
      v[4 * h + 2] = make_float2(lo_f(t.z), hi_f(t.z));
      v[4 * h + 3] = make_float2(lo_f(t.w), hi_f(t.w));
    }
  }
}

// Sum over a unit's columns of four row sums a lane: lane l gets row l's.
__device__ __forceinline__ float fold_rows(const float (&s)[4], int lane) {
  const bool a = (lane & 1) != 0, b = (lane & 2) != 0;
  const float x = (a ? s[1] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, a ? s[0] : s[1], 1);
  const float y = (a ? s[3] : s[2]) + __shfl_xor_sync(0xFFFFFFFFu, a ? s[2] : s[3], 1);
  return (b ? y : x) + __shfl_xor_sync(0xFFFFFFFFu, b ? x : y, 2);
}

}  // namespace mx
