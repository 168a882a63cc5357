// MXFP4 on gfx950: the layout of a matrix held in it and the conversions of a
// block's elements, shared by the quantising kernels and the products.
//
// Codes: row-major, 16 bytes per block of 32 columns, two a byte, the first in the
// low half: one block is one lane's operand of v_mfma_scale_f32_16x16x128_f8f6f4.
// Scales: E8M0 bytes in the order in which that instruction's operands want them.
// A lane (q, g) = 16 g + q holds row q of a tile of 16 and, in step s of four, block
// 4 s + g of 16; so 16 rows x 16 blocks take 256 bytes, that of (q, 4 s + g) at
// 4 (16 g + q) + s: a wave's load of 64 dwords brings the scales of four steps,
// whole lines, and the instruction picks the byte.  Rows and blocks are filled up
// to 16 with byte 0 (2^-127; never 255, whose NaN a zero code would not hide).
#pragma once

#include "common.hpp"

namespace qn {

constexpr int kMxBlock = 32;

__host__ __device__ inline int64_t mx_blocks(int64_t cols) { return (cols + 31) / 32; }
__host__ __device__ inline int64_t mx_chunks(int64_t cols) { return (cols + 511) / 512; }   // 16 blocks each
__host__ __device__ inline int64_t mx_code_bytes(int64_t rows, int64_t cols) { return rows * mx_blocks(cols) * 16; }
__host__ __device__ inline int64_t mx_scale_bytes(int64_t rows, int64_t cols) {
  return (rows + 15) / 16 * mx_chunks(cols) * 256;
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// E8M0 byte of a block whose largest magnitude has the fp32 bits `top`:
// floor(log2) - 2, at least -127, biased by 127; 255 where top is not finite.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// The codes of eight values of a type; zeros where the block's byte is 255.  The
// instructions round to nearest, ties to even codes, past 6 to 6, and take only
// the exponent of the scale (checked against the definition for every 16-bit value).
__device__ __forceinline__ uint32_t mx_keep(uint32_t codes, uint32_t byte) { return byte == 255u ? 0u : codes; }
__device__ __forceinline__ uint32_t mx_codes8(Bf16, const uint4& v, uint32_t byte) {
  const float s = mx_scale(byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v.x), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v.y), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v.z), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v.w), s, 3);
  return mx_keep(w, byte);
}
__device__ __forceinline__ uint32_t mx_codes8(F16, const uint4& v, uint32_t byte) {
  const float s = mx_scale(byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, v.x), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, v.y), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, v.z), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, v.w), s, 3);
  return mx_keep(w, byte);
}
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], uint32_t byte) {
  const float s = mx_scale(byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
  return mx_keep(w, byte);
}

// fp32 bits of the largest magnitude, from the largest of the 16-bit magnitudes
// (ordered as integers; an infinity or a NaN comes out with exponent 255).
__device__ __forceinline__ uint32_t mx_widen_top(Bf16, uint32_t m) { return m << 16; }
__device__ __forceinline__ uint32_t mx_widen_top(F16, uint32_t m) {
  return __builtin_bit_cast(uint32_t, F16::widen(m));
}

// Byte b (0 .. 3) of a word of codes as two 16-bit values; a scale byte of 255
// gives NaN.
template <int b>
__device__ __forceinline__ uint32_t mx_pair(Bf16, uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, b));
}
template <int b>
__device__ __forceinline__ uint32_t mx_pair(F16, uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, b));
}
template <class T>
__device__ __forceinline__ uint4 mx_values8(uint32_t w, float s) {
  return make_uint4(mx_pair<0>(T{}, w, s), mx_pair<1>(T{}, w, s), mx_pair<2>(T{}, w, s), mx_pair<3>(T{}, w, s));
}
__device__ __forceinline__ void mx_values8(uint32_t w, float s, float (&v)[8]) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
  const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
  v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
}

}  // namespace qn
