// Device-side arithmetic of the 8-bit activation checkpoints (act8.hip says
// what they are), shared with the kernels that write or read them on the way.
#pragma once

#include "common.hpp"

namespace qn {

// Largest magnitude of two pairs of 16-bit floats: without their signs the
// bit patterns order like the values (infinity and NaN above every number).
__device__ __forceinline__ uint32_t act8_max2(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t act8_max4(const uint4& v) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  return act8_max2(act8_max2(v.x & kAbs, v.y & kAbs), act8_max2(v.z & kAbs, v.w & kAbs));
}

// The same over a block that eight neighbouring lanes hold, 8 values each.
__device__ __forceinline__ uint32_t act8_block_max(const uint4& v) {
  uint32_t m = act8_max4(v);
  m = act8_max2(m, __shfl_xor(m, 1, 64));
  m = act8_max2(m, __shfl_xor(m, 2, 64));
  m = act8_max2(m, __shfl_xor(m, 4, 64));
  return max(m & 0xffffu, m >> 16);
}

// What encoding a block needs of its largest magnitude (16-bit pattern).
struct Act8Scale {
  float k, a, inv;   // quotient = (k x) / a, both scaled by a power of two into fp32's middle; inv ~ 1 / a
  uint16_t kept;     // the stored magnitude; NaN where the block is not finite
};

template <class T>
__device__ __forceinline__ Act8Scale act8_scale(uint32_t amax) {
  constexpr uint32_t kInf = T::kDtype == Bf16::kDtype ? 0x7f80u : 0x7c00u;
  Act8Scale s;
  const bool bad = amax >= kInf;
  const float a = T::widen(amax);
  // |x| <= a: the product and the reciprocal stay normal numbers after this
  const float sc = a > 0x1p64f ? 0x1p-64f : (a < 0x1p-64f ? 0x1p64f : 1.0f);
  const bool none = bad || amax == 0;
  s.k = none ? 0.0f : 127.0f * sc;
  s.a = none ? 1.0f : a * sc;
  s.inv = __builtin_amdgcn_rcpf(s.a);
  s.kept = static_cast<uint16_t>(bad ? 0x7fffu : amax);
  return s;
}

// Code of x: RNE(k x / a), in the low byte (two's complement).  Adding
// 1.5 * 2^23 leaves the rounded integer in the low bits.
__device__ __forceinline__ uint32_t act8_code(float x, const Act8Scale& s) {
  const float t = x * s.k;                                  // exact: 11 bits times 7
  const float q1 = t * s.inv;
  const float q = __builtin_fmaf(__builtin_fmaf(-q1, s.a, t), s.inv, q1);
  return __builtin_bit_cast(uint32_t, q + 12582912.0f);
}

__device__ __forceinline__ uint32_t act8_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
  return lo | hi;
}

template <class T>
__device__ __forceinline__ uint32_t act8_codes4(uint32_t p0, uint32_t p1, const Act8Scale& s) {
  float x[4] = {T::widen(p0 & 0xffffu), T::widen(p0 >> 16), T::widen(p1 & 0xffffu), T::widen(p1 >> 16)};
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a block that is not finite has k = 0; 0 * inf must still give code 0
    q[i] = act8_code(s.k == 0.0f ? 0.0f : x[i], s);
  }
  return act8_pack4(q[0], q[1], q[2], q[3]);
}
template <class T>
__device__ __forceinline__ uint2 act8_codes8(const uint4& v, const Act8Scale& s) {
  return make_uint2(act8_codes4<T>(v.x, v.y, s), act8_codes4<T>(v.z, v.w, s));
}

// fl32(a / 127) of a stored magnitude.
template <class T>
__device__ __forceinline__ float act8_step(uint32_t kept) {
  return __fdiv_rn(T::widen(kept), 127.0f);
}
// Four codes (one per byte) -> four 16-bit values.  (In fp16 the product may be
// rounded once, in its conversion, or twice: no code and magnitude tell them apart.)
template <class T>
__device__ __forceinline__ uint2 act8_values4(uint32_t q, float step) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(static_cast<float>(static_cast<int8_t>(q >> (8 * i))), step);
  return make_uint2(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]));
}

}  // namespace qn
