// The quantising of one 16 x 512 piece of a matrix into MXFP4, for the kernel that does
// only that (mxfp4.hip) and for the one in front of the products (mx_gemv.hip).
#pragma once

#include "act8.hpp"
#include "common.hpp"
#include "mxfp4.hpp"

namespace qn {

namespace {

struct MxArgs {
  const void* x;        // quantise: input; dequantise: output (written)
  int64_t ld;           // its row stride, elements
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, cols;   // of the MXFP4 matrix
  int64_t chunks;       // mx_chunks(cols)
};

// Eight neighbouring elements of a row in a lane.
struct F32 {};
template <class T>
struct Row8 {
  uint4 v = make_uint4(0, 0, 0, 0);
  __device__ void load(const void* x, int64_t at) { v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at); }
  __device__ uint32_t top() const {
    const uint32_t m = act8_max4(v);
    return max(m & 0xffffu, m >> 16);
  }
  __device__ static uint32_t widen(uint32_t m) { return mx_widen_top(T{}, m); }
  __device__ uint32_t codes(uint32_t byte) const { return mx_codes8(T{}, v, byte); }
};
template <>
struct Row8<F32> {
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  __device__ void load(const void* x, int64_t at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
    return m;
  }
  __device__ static uint32_t widen(uint32_t m) { return m; }
  __device__ uint32_t codes(uint32_t byte) const { return mx_codes8(v, byte); }
};

// A workgroup's piece: rows 16 tile .. +15, columns 512 chunk .. +511; a wave four of the rows.
template <class T>
__device__ __forceinline__ void mx_quantize_piece(const MxArgs& a, int64_t piece) {
  const int64_t tile = piece / a.chunks, chunk = piece - tile * a.chunks;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = tile * 16 + 4 * wave, col = chunk * 512 + 8 * lane;
  const int64_t stride = mx_blocks(a.cols) * 16;
  Row8<T> v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + i < a.rows && col < a.cols) v[i].load(a.x, (row0 + i) * a.ld + col);
  uint32_t word[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t m = v[i].top();
    m = max(m, static_cast<uint32_t>(__shfl_xor(m, 1, 64)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(m, 2, 64)));
    const uint32_t byte = mx_scale_byte(Row8<T>::widen(m));
    const uint32_t q = v[i].codes(byte);
    if (row0 + i < a.rows && (col >> 5) * 16 < stride)
      *reinterpret_cast<uint32_t*>(a.codes + (row0 + i) * stride + chunk * 256 + 4 * lane) = q;
    // the bytes of blocks g, 4 + g, 8 + g, 12 + g into one word, in the lanes of g
    uint32_t w = byte << (8 * (lane >> 4));
    w |= __shfl_xor(w, 16, 64);
    word[i] = w | __shfl_xor(w, 32, 64);
  }
  if (lane < 16 && (lane & 3) == 0)
    *reinterpret_cast<uint4*>(a.scales + piece * 256 + 4 * (16 * (lane >> 2) + 4 * wave)) =
        make_uint4(word[0], word[1], word[2], word[3]);
}

}  // namespace

}  // namespace qn
