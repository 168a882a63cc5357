// 8-bit checkpoints of 16-bit activations, for gfx950: encode and decode.
//
// Per row, blocks of 64 consecutive columns (the last one may be shorter):
//   a  = max |x| of the block, itself one of the 16-bit values, so kept exactly;
//   q  = nearest integer to 127 x / a, ties to even (0 where a = 0);
//   x^ = RNE_16(fl32(q * fl32(a / 127))).
// A block that holds an infinity or a NaN keeps a = NaN and decodes to NaN
// throughout, so a checkpoint never hides an overflow.
//
// Both passes are bound by memory: 2 bytes read and 1.03 written per element
// (decode: the other way round).  Eight lanes own a block: one 16-byte load of
// eight values a lane, three exchanges for the maximum, one 8-byte store of
// codes; kU such loads are in flight a lane.
// The quotient costs two products and two fused operations: with r = rcp(a)
// (one ulp off at most) the estimate t r is corrected by its exact remainder,
// which makes a quotient that fp32 holds exactly come out exactly - so ties
// round to even - and leaves the others within an ulp.  127 x / a of two
// 16-bit values is either a tie or at least 2^-19 of itself away from one
// (their significands have at most 11 bits), so every code is the exact one.
#include "act8.hpp"
#include "common.hpp"
#include "kernels.hpp"

namespace qn {

namespace {

constexpr int kThreads = 256;
#ifndef QN_A8_U
#define QN_A8_U 4
#endif
constexpr int kU = QN_A8_U;          // chunks of 8 values in flight per lane
#ifndef QN_A8_GRID
#define QN_A8_GRID 2048
#endif
constexpr int64_t kGrid = QN_A8_GRID;   // most workgroups (8 per CU); larger tensors loop

struct A8Args {
  const uint16_t* x;     // encode: input; decode: output (written)
  int64_t ld;            // its row stride, elements
  int8_t* codes;         // rows x cols
  uint16_t* absmax;      // rows x nb
  uint32_t cols, nb;     // nb = ceil(cols / 64)
  uint32_t slots;        // rows * nb * 8 chunks of 8 columns
};

// Chunk slot -> row and first column.  flat: cols % 64 == 0 and ld == cols, so
// every offset is linear in the slot and needs no division.
template <bool kFlat>
__device__ __forceinline__ void slot_place(const A8Args& a, uint32_t s, uint32_t& row, uint32_t& col) {
  if (kFlat) {
    row = 0;
    col = s * 8;
  } else {
    const uint32_t per = a.nb * 8;
    row = s / per;
    col = (s - row * per) * 8;
  }
}

template <class T, bool kFlat>
__global__ __launch_bounds__(kThreads) void act8_encode_kernel(A8Args a) {
  const uint32_t step = gridDim.x * (kThreads * kU);
  for (uint32_t base = blockIdx.x * (kThreads * kU); base < a.slots; base += step) {
    uint4 v[kU];
    uint32_t row[kU], col[kU];
    bool ok[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t s = base + u * kThreads + threadIdx.x;
      slot_place<kFlat>(a, s, row[u], col[u]);
      ok[u] = s < a.slots && (kFlat || col[u] < a.cols);
      v[u] = make_uint4(0, 0, 0, 0);
      if (ok[u]) v[u] = *reinterpret_cast<const uint4*>(a.x + row[u] * a.ld + col[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      // every lane of the block's eight takes part: a chunk past the row's end counts as zeros
      const Act8Scale sc = act8_scale<T>(act8_block_max(v[u]));
      const uint2 q = act8_codes8<T>(v[u], sc);
      if (!ok[u]) continue;
      *reinterpret_cast<uint2*>(a.codes + static_cast<int64_t>(row[u]) * a.cols + col[u]) = q;
      if ((col[u] & 63u) == 0) a.absmax[static_cast<int64_t>(row[u]) * a.nb + (col[u] >> 6)] = sc.kept;
    }
  }
}

template <class T, bool kFlat>
__global__ __launch_bounds__(kThreads) void act8_decode_kernel(A8Args a) {
  const uint32_t step = gridDim.x * (kThreads * kU);
  for (uint32_t base = blockIdx.x * (kThreads * kU); base < a.slots; base += step) {
    uint2 q[kU];
    uint32_t row[kU], col[kU], am[kU];
    bool ok[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t s = base + u * kThreads + threadIdx.x;
      slot_place<kFlat>(a, s, row[u], col[u]);
      ok[u] = s < a.slots && (kFlat || col[u] < a.cols);
      q[u] = make_uint2(0, 0);
      am[u] = 0;
      if (ok[u]) {
        q[u] = *reinterpret_cast<const uint2*>(a.codes + static_cast<int64_t>(row[u]) * a.cols + col[u]);
        am[u] = a.absmax[static_cast<int64_t>(row[u]) * a.nb + (col[u] >> 6)];
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (!ok[u]) continue;
      const float step8 = act8_step<T>(am[u]);
      const uint2 lo = act8_values4<T>(q[u].x, step8), hi = act8_values4<T>(q[u].y, step8);
      *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.x) + row[u] * a.ld + col[u]) =
          make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

A8Args a8_args(int64_t rows, int64_t cols, const uint16_t* x, int64_t ld, int8_t* codes, uint16_t* absmax) {
  const int64_t nb = (cols + 63) / 64;
  return A8Args{x, ld, codes, absmax, static_cast<uint32_t>(cols), static_cast<uint32_t>(nb),
                static_cast<uint32_t>(rows * nb * 8)};
}
unsigned a8_grid(const A8Args& a) {
  const int64_t g = (static_cast<int64_t>(a.slots) + kThreads * kU - 1) / (kThreads * kU);
  return static_cast<unsigned>(g < kGrid ? g : kGrid);
}

}  // namespace

hipError_t launch_act8_encode(int64_t rows, int64_t cols, const uint16_t* X, int64_t ld, int8_t* codes,
                              uint16_t* absmax, hipStream_t stream, int dtype) {
  const A8Args a = a8_args(rows, cols, X, ld, codes, absmax);
  const bool flat = cols % 64 == 0 && ld == cols;
  auto* k = dtype == kDtypeF16 ? (flat ? act8_encode_kernel<F16, true> : act8_encode_kernel<F16, false>)
                               : (flat ? act8_encode_kernel<Bf16, true> : act8_encode_kernel<Bf16, false>);
  Timer tm(QK_ACT8_ENCODE, stream);
  hipLaunchKernelGGL(k, dim3(a8_grid(a)), dim3(kThreads), 0, stream, a);
  tm.stop();
  return hipGetLastError();
}

hipError_t launch_act8_decode(int64_t rows, int64_t cols, const int8_t* codes, const uint16_t* absmax, uint16_t* X,
                              int64_t ld, hipStream_t stream, int dtype) {
  const A8Args a = a8_args(rows, cols, X, ld, const_cast<int8_t*>(codes), const_cast<uint16_t*>(absmax));
  const bool flat = cols % 64 == 0 && ld == cols;
  auto* k = dtype == kDtypeF16 ? (flat ? act8_decode_kernel<F16, true> : act8_decode_kernel<F16, false>)
                               : (flat ? act8_decode_kernel<Bf16, true> : act8_decode_kernel<Bf16, false>);
  Timer tm(QK_ACT8_DECODE, stream);
  hipLaunchKernelGGL(k, dim3(a8_grid(a)), dim3(kThreads), 0, stream, a);
  tm.stop();
  return hipGetLastError();
}

}  // namespace qn
