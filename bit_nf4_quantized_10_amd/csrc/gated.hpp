// The activation of the gated feed-forward block and what its kernels keep:
// H = act(G) * U and, for the backward, dG = dH U act'(G), dU = dH act(G).
#pragma once

#include "act8.hpp"
#include "common.hpp"

namespace qn {

// Where a forward keeps G and U (M x 2F, [G | U]): in 16 bits, in 8, or not.
struct GatedKeep {
  uint16_t* gu = nullptr;
  int8_t* codes = nullptr;      // M x 2F
  uint16_t* absmax = nullptr;   // M x 2F / 64
};

// Sigmoid of y by the hardware's 2^x and reciprocal (about 1e-7 relative);
// e^-y overflows to infinity and gives 0.
__device__ __forceinline__ float sigmoid_of(float y) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(y * -1.44269504f));
}

// Both activations are g sigmoid(y): silu with y = g, gelu (its tanh form
// 0.5 g (1 + tanh(y / 2))) with y = 2 sqrt(2 / pi) (g + 0.044715 g^3).
// The derivative is s + g s (1 - s) y'.  Past |g| = 1000 the sigmoid is 0 or 1
// in fp32, so g is clamped there before the cube, and -inf (what fp16 keeps of a
// G below -65504) is taken as the lowest finite number: no infinity meets a zero.
constexpr float kGelu0 = 1.5957691216f, kGelu1 = 0.044715f;
__device__ __forceinline__ float clamp_g(float g) {
  return __builtin_fabsf(g) > 1000.0f ? __builtin_copysignf(1000.0f, g) : g;   // a NaN stays one
}
__device__ __forceinline__ float gelu_y(float g) {
  const float x = clamp_g(g);
  return kGelu0 * x * __builtin_fmaf(kGelu1 * x, x, 1.0f);
}
__device__ __forceinline__ float above_inf(float g) { return g == -__builtin_inff() ? -3.40282347e38f : g; }
template <bool kGelu>
__device__ __forceinline__ float act_of(float g) {
  return above_inf(g) * sigmoid_of(kGelu ? gelu_y(g) : g);
}
// f = act(g), df = act'(g)
template <bool kGelu>
__device__ __forceinline__ void act_grad_of(float g, float& f, float& df) {
  const float s = sigmoid_of(kGelu ? gelu_y(g) : g);
  const float x = clamp_g(g);
  const float dy = kGelu ? kGelu0 * __builtin_fmaf(3.0f * kGelu1 * x, x, 1.0f) : 1.0f;
  f = above_inf(g) * s;
  df = __builtin_fmaf(x * s * (1.0f - s), dy, s);
}

// 8 consecutive columns (a chunk) of one row: H and what is kept, from G and U
// in fp32.  Eight neighbouring lanes hold one 64-column block.
template <class T, bool kGelu>
__device__ __forceinline__ void gated_store8(const float (&g)[8], const float (&u)[8], int64_t m, int64_t col, int64_t F,
                                             uint16_t* H, const GatedKeep& keep) {
  if (H != nullptr) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_of<kGelu>(g[e]) * u[e];
    *reinterpret_cast<uint4*>(H + m * F + col) =
        make_uint4(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]), T::pack2(v[6], v[7]));
  }
  if (keep.gu == nullptr && keep.codes == nullptr) return;
  const uint4 g16 = make_uint4(T::pack2(g[0], g[1]), T::pack2(g[2], g[3]), T::pack2(g[4], g[5]), T::pack2(g[6], g[7]));
  const uint4 u16 = make_uint4(T::pack2(u[0], u[1]), T::pack2(u[2], u[3]), T::pack2(u[4], u[5]), T::pack2(u[6], u[7]));
  if (keep.gu != nullptr) {
    *reinterpret_cast<uint4*>(keep.gu + m * 2 * F + col) = g16;
    *reinterpret_cast<uint4*>(keep.gu + m * 2 * F + F + col) = u16;
    return;
  }
  const int64_t nb = F / 64;
  const Act8Scale sg = act8_scale<T>(act8_block_max(g16)), su = act8_scale<T>(act8_block_max(u16));
  *reinterpret_cast<uint2*>(keep.codes + m * 2 * F + col) = act8_codes8<T>(g16, sg);
  *reinterpret_cast<uint2*>(keep.codes + m * 2 * F + F + col) = act8_codes8<T>(u16, su);
  if ((col & 63) == 0) {
    keep.absmax[m * 2 * nb + col / 64] = sg.kept;
    keep.absmax[m * 2 * nb + nb + col / 64] = su.kept;
  }
}

}  // namespace qn
