// MXFP4 quantisation and its inverse, for gfx950.  Per row, blocks of 32 columns
// (the last one filled up with zeros):
//   s = max(-127, floor(log2 max|x|) - 2),  code = the nearest of the E2M1 values
//   0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives to x / 2^s (ties to the even
//   code, past 6 the last one, the sign kept), value = code's * 2^s.
// A block holding an infinity or a NaN has scale byte 255 and decodes to NaN.
// Nothing is rounded but the elements themselves: the scale is a power of two.
//
// All passes are bound by memory (2 or 4 bytes read and 0.53 written an element, or
// the other way round).  A workgroup takes one 16 x 512 piece, whose 256 scale bytes
// (mxfp4.hpp) are then its own whole lines; a lane loads 8 columns, four lanes hold
// a block.  11008 x 4096 is quantised in 38 us from fp32 (5.3 TB/s) and 21 from bf16, and
// dequantised in 38 and 23; a large copy runs at 5.1 TB/s.  Across (a K x N weight quantised along K) a lane holds 32 elements of
// one or two columns, so a block is one lane's, and the codes turn in LDS.
#include "common.hpp"
#include "kernels.hpp"
#include "mx_quant.hpp"

namespace qn {

namespace {

constexpr int kThreads = 256;

template <class T>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(MxArgs a) {
  mx_quantize_piece<T>(a, blockIdx.x);
}

// A lane: 8 columns of 16 bits, or 4 and 4 of fp32 256 apart, so that its stores and its
// neighbours' are whole lines (8 together: 52 us for 4096 x 11008 instead of 40).
template <class T>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(MxArgs a) {
  constexpr int kParts = __is_same(T, F32) ? 2 : 1, kCols = 8 / kParts;
  const int64_t tile = blockIdx.x / a.chunks, chunk = blockIdx.x - tile * a.chunks;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = tile * 16 + 4 * wave;
  const int64_t stride = mx_blocks(a.cols) * 16;
  uint32_t q[kParts][4];
  uint4 sw[kParts];
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
    const int col = kCols * (64 * h + lane), b = col >> 5;   // of the 512
    if (chunk * 512 + col >= a.cols) continue;
    sw[h] = *reinterpret_cast<const uint4*>(a.scales + blockIdx.x * int64_t(256) + 4 * (16 * (b & 3) + 4 * wave));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[h][i] = row0 + i < a.rows ? *reinterpret_cast<const uint32_t*>(a.codes + (row0 + i) * stride + chunk * 256 + 4 * (col >> 3)) : 0u;
  }
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
    const int col = kCols * (64 * h + lane), b = col >> 5;
    if (chunk * 512 + col >= a.cols) continue;
    const uint32_t word[4] = {sw[h].x, sw[h].y, sw[h].z, sw[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (row0 + i >= a.rows) continue;
      const float s = mx_scale((word[i] >> (8 * (b >> 2))) & 255u);
      const int64_t at = (row0 + i) * a.ld + chunk * 512 + col;
      if constexpr (__is_same(T, F32)) {
        const uint32_t w = q[h][i] >> (16 * (lane & 1));
        const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
        *reinterpret_cast<float4*>(static_cast<float*>(const_cast<void*>(a.x)) + at) = make_float4(lo[0], lo[1], hi[0], hi[1]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(const_cast<void*>(a.x)) + at) = mx_values8<T>(q[h][i], s);
      }
    }
  }
}

// Across: x is cols x rows (row stride ld).  Workgroup: 64 of its columns, 512 of its
// rows; wave w blocks 4 w .. +3.  The codes of row n's block b lie in LDS at chunk
// b ^ (n & 15) of its 256 bytes, so that neither side of the turn meets on a bank.
// Neighbours in x are neighbours in the grid, and x, read once, is not kept: 4096 x 11008
// of fp32 40 us (5.2 TB/s), of bf16 23 us; chunk by chunk 48 and 28, kept 45 and 26.
constexpr int kTurnRows = 64;
template <class T>
__global__ __launch_bounds__(kThreads) void mx_quantize_across_kernel(MxArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t sc[kTurnRows * 256];
  __shared__ __attribute__((aligned(16))) uint8_t ss[kTurnRows * 16];
  const int64_t panels = gridDim.x / a.chunks, chunk = blockIdx.x / panels, panel = blockIdx.x - chunk * panels;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t n0 = panel * kTurnRows, k0 = chunk * 512;
  auto put = [&](int n, int b, const uint4& codes, uint32_t byte) {
    *reinterpret_cast<uint4*>(sc + n * 256 + ((b ^ (n & 15)) << 4)) = codes;
    ss[(n >> 4) * 256 + 4 * (16 * (b & 3) + (n & 15)) + (b >> 2)] = static_cast<uint8_t>(byte);
  };
  if constexpr (__is_same(T, F32)) {
    const int64_t n = n0 + lane;
    const float* x = static_cast<const float*>(a.x) + n;
    for (int j = 0; j < 4; ++j) {
      const int b = 4 * wave + j;
      const int64_t k = k0 + 32 * b;
      float v[32];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = n < a.rows && k + i < a.cols ? __builtin_nontemporal_load(x + (k + i) * a.ld) : 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
      const uint32_t byte = mx_scale_byte(m);
      uint32_t w[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float e[8] = {v[8 * p], v[8 * p + 1], v[8 * p + 2], v[8 * p + 3], v[8 * p + 4], v[8 * p + 5], v[8 * p + 6], v[8 * p + 7]};
        w[p] = mx_codes8(e, byte);
      }
      put(lane, b, make_uint4(w[0], w[1], w[2], w[3]), byte);
    }
  } else {
    // two columns a lane, two blocks a wave at a time
    const int c = 2 * (lane & 31);
    const int64_t n = n0 + c;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + n;
    for (int j = 0; j < 2; ++j) {
      const int b = 4 * wave + 2 * j + (lane >> 5);
      const int64_t k = k0 + 32 * b;
      uint32_t v[32], m = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) 
        v[i] = n < a.rows && k + i < a.cols ? __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(x + (k + i) * a.ld)) : 0u;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = act8_max2(m, v[i] & 0x7fff7fffu);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t byte = mx_scale_byte(mx_widen_top(T{}, h ? m >> 16 : m & 0xffffu));
        const uint32_t sel = h ? 0x07060302u : 0x05040100u;
        uint32_t w[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint32_t e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = __builtin_amdgcn_perm(v[8 * p + 2 * i + 1], v[8 * p + 2 * i], sel);
          w[p] = mx_codes8(T{}, make_uint4(e[0], e[1], e[2], e[3]), byte);
        }
        put(c + h, b, make_uint4(w[0], w[1], w[2], w[3]), byte);
      }
    }
  }
  __syncthreads();
  const int64_t nb = mx_blocks(a.cols);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int at = u * kThreads + t, n = at >> 4, b = at & 15;
    if (n0 + n < a.rows && 16 * chunk + b < nb)
      *reinterpret_cast<uint4*>(a.codes + ((n0 + n) * nb + 16 * chunk + b) * 16) =
          *reinterpret_cast<const uint4*>(sc + n * 256 + ((b ^ (n & 15)) << 4));
  }
  if (lane < 16) {   // wave: one tile of 16 rows
    const int64_t tile = panel * 4 + wave;
    if (tile * 16 < a.rows)
      *reinterpret_cast<uint4*>(a.scales + (tile * a.chunks + chunk) * 256 + 16 * lane) =
          *reinterpret_cast<const uint4*>(ss + wave * 256 + 16 * lane);
  }
}

// Its inverse: 128 rows of the matrix by 512 columns, into x (cols x rows).  A lane
// turns an 8 x 8 block: eight words of codes (chunks in LDS at c ^ (row >> 3), so
// that 16 lanes' reads fall on different banks) into eight 16- or 32-byte stores.
// 11008 x 4096: 43 us into fp32 (4.7 TB/s), 23.5 into bf16; neighbours in x together, as
// above, gained 3 % in fp32 and lost 3 % in bf16.
constexpr int kBackRows = 128;
template <class T>
__global__ __launch_bounds__(kThreads) void mx_dequantize_across_kernel(MxArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t sc[kBackRows * 256];
  __shared__ __attribute__((aligned(16))) uint8_t ss[kBackRows * 16];
  const int64_t panel = blockIdx.x / a.chunks, chunk = blockIdx.x - panel * a.chunks;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t n0 = panel * kBackRows, k0 = chunk * 512, nb = mx_blocks(a.cols);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int at = u * kThreads + t, n = at >> 4, b = at & 15;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n0 + n < a.rows && 16 * chunk + b < nb) v = *reinterpret_cast<const uint4*>(a.codes + ((n0 + n) * nb + 16 * chunk + b) * 16);
    *reinterpret_cast<uint4*>(sc + n * 256 + ((b ^ (n >> 3)) << 4)) = v;
  }
  if (t < kBackRows) {   // 16 bytes a thread
    const int64_t tile = panel * 8 + (t >> 4);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (tile * 16 < a.rows) v = *reinterpret_cast<const uint4*>(a.scales + (tile * a.chunks + chunk) * 256 + 16 * (t & 15));
    *reinterpret_cast<uint4*>(ss + t * 16) = v;
  }
  __syncthreads();
  const int ng = lane & 15;   // rows 8 ng .. +7
  const int64_t n = n0 + 8 * ng;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int ko = 16 * u + 4 * wave + (lane >> 4), b = ko >> 2;   // columns 8 ko .. +7, in block b
    const int64_t k = k0 + 8 * ko;
    if (k >= a.cols || n >= a.rows) continue;
    uint32_t q[8];
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 8 * ng + i;
      q[i] = *reinterpret_cast<const uint32_t*>(sc + row * 256 + ((b ^ ng) << 4) + 4 * (ko & 3));
      s[i] = mx_scale(ss[(row >> 4) * 256 + 4 * (16 * (b & 3) + (row & 15)) + (b >> 2)]);
    }
    if constexpr (__is_same(T, F32)) {
      float v[8][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) mx_values8(q[i], s[i], v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float4* out = reinterpret_cast<float4*>(static_cast<float*>(const_cast<void*>(a.x)) + (k + j) * a.ld + n);
        out[0] = make_float4(v[0][j], v[1][j], v[2][j], v[3][j]);
        out[1] = make_float4(v[4][j], v[5][j], v[6][j], v[7][j]);
      }
    } else {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mx_values8<T>(q[i], s[i]);
      auto word = [](const uint4& w, int i) { return i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w)); };
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
        uint32_t d[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) d[p] = __builtin_amdgcn_perm(word(v[2 * p + 1], j >> 1), word(v[2 * p], j >> 1), sel);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(const_cast<void*>(a.x)) + (k + j) * a.ld + n) =
            make_uint4(d[0], d[1], d[2], d[3]);
      }
    }
  }
}

// The kernel of an element type (NF4_OUT_*).
template <class K>
auto pick(int type, K bf16, K f16, K f32) {
  return type == NF4_OUT_BF16 ? bf16 : (type == NF4_OUT_F16 ? f16 : f32);
}

}  // namespace

hipError_t launch_mx_quantize(int type, bool across, const void* X, int64_t ld, MxView m, hipStream_t stream) {
  const MxArgs a{X, ld, m.codes, m.scales, m.rows, m.cols, mx_chunks(m.cols)};
  const int64_t panels = (m.rows + (across ? kTurnRows : 16) - 1) / (across ? kTurnRows : 16);
  auto* k = across ? pick(type, mx_quantize_across_kernel<Bf16>, mx_quantize_across_kernel<F16>, mx_quantize_across_kernel<F32>)
                   : pick(type, mx_quantize_kernel<Bf16>, mx_quantize_kernel<F16>, mx_quantize_kernel<F32>);
  Timer tm(QK_MX_QUANT, stream);
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(panels * a.chunks)), dim3(kThreads), 0, stream, a);
  tm.stop();
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(int type, bool across, MxView m, void* X, int64_t ld, hipStream_t stream) {
  const MxArgs a{X, ld, m.codes, m.scales, m.rows, m.cols, mx_chunks(m.cols)};
  const int64_t panels = (m.rows + (across ? kBackRows : 16) - 1) / (across ? kBackRows : 16);
  auto* k = across ? pick(type, mx_dequantize_across_kernel<Bf16>, mx_dequantize_across_kernel<F16>, mx_dequantize_across_kernel<F32>)
                   : pick(type, mx_dequantize_kernel<Bf16>, mx_dequantize_kernel<F16>, mx_dequantize_kernel<F32>);
  Timer tm(QK_MX_DEQUANT, stream);
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(panels * a.chunks)), dim3(kThreads), 0, stream, a);
  tm.stop();
  return hipGetLastError();
}

}  // namespace qn
