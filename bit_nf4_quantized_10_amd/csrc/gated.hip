// The gated feed-forward front of the layer for more than 16 rows, on gfx950:
//   [Zg | Zu] = X A,  G = X Ŵg + c Zg Bg,  U = X Ŵu + c Zu Bu,  H = act(G) * U
// and the elementwise half of its backward.  (Up to 16 rows: gemv.hip.)
//
// Forward: one dense GEMM over both weights, dequantized beforehand and stacked
// (2F x K).  A 256 x 256 tile of it takes 128 columns of each weight (Dense's
// kGated), so the lane that holds G of an element also holds its U: the
// activation, the product, the 16-bit rounding and, where the backward wants
// G and U kept in 8 bits, the checkpoint's encoding run on the accumulators,
// and neither G nor U passes through memory to be combined.  Bound by the
// matrix cores, as the GEMM it is made of.
// With few tiles the reduction is split (plan_split) and the fp32 partials are
// summed in split order by gated_sum_kernel, which then does the same.
//
// Backward: dG = dH U act'(G), dU = dH act(G) (gated_dy_kernel, bound by
// memory: 2 bytes of dH, 4 or 2.06 of G and U, 4 written per element), stored
// side by side as the M x 2F gradient of a grouped linear; the rest is that
// linear's backward (layer.hip).  G and U that were not kept are computed
// again by the forward's own kernels.
#include <hip/hip_ext.h>

#include "gated.hpp"
#include "gemm_core.hpp"

namespace qn {

namespace {

struct GatedArgs {
  BigArgs g;        // N = 2F, ext_a = [hi | lo] of c Z (M x 4r), ext_b = Bᵀ (2F x r), out = H (may be null)
  GatedKeep keep;
  int64_t F;
};

enum { kKeepNone = 0, kKeep16 = 1, kKeep8 = 2 };

// 64 columns of one weight at one output row, held by lanes l and l ^ 32
// (8 columns each step, 4 per lane): their checkpoint.  pairs[2 t], pairs[2 t + 1]:
// the 16-bit values of the lane's t-th group of 4.  Returns the 4-byte codes.
template <class T>
__device__ __forceinline__ uint16_t encode_block(const uint32_t (&pairs)[16], uint32_t (&codes)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = act8_max2(m, pairs[i] & 0x7fff7fffu);
  m = act8_max2(m, __shfl_xor(m, 32, 64));
  const Act8Scale s = act8_scale<T>(max(m & 0xffffu, m >> 16));
#pragma unroll
  for (int t = 0; t < 8; ++t) codes[t] = act8_codes4<T>(pairs[2 * t], pairs[2 * t + 1], s);
  return s.kept;
}

// The tile's epilogue.  Lane l holds, for tiles (i, j) and (i, j + 2), row
// 32i + l%32 and columns wn*64 + 32j + 8jj + 4(l/32) .. +3 of G and U.
template <class T, bool kGelu, int kKeep, class Core>
__device__ __forceinline__ void finish_gated(const Core& k, const GatedArgs& p, f32x16 (&acc)[4][4]) {
  const BigArgs& a = p.g;
  const int lane = k.lane, r32 = lane & 31, h = lane >> 5, wm = k.wave >> 1, wn = k.wave & 1;
  const int64_t F = p.F;
  char* st = k.smem;
  if constexpr (kKeep == kKeep16) {
    // [G | U] as 16-bit rows of 256 columns: chunk q < 16 of G, the others of U
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int R = wm * 128 + 32 * i + r32;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int q = (j >> 1) * 16 + wn * 8 + 4 * (j & 1) + jj;
          uint2 v;
          v.x = T::pack2(acc[i][j][4 * jj], acc[i][j][4 * jj + 1]);
          v.y = T::pack2(acc[i][j][4 * jj + 2], acc[i][j][4 * jj + 3]);
          *reinterpret_cast<uint2*>(st + R * 512 + ((q ^ r32) << 4) + 8 * h) = v;
        }
    }
    __syncthreads();
    const int q = lane & 31;
    const int64_t col = k.c0 + 8 * (q & 15);
#pragma unroll 4
    for (int u = 0; u < 32; ++u) {
      const int R = k.wave * 64 + 2 * u + (lane >> 5);
      const int64_t m = k.m0 + R;
      const uint4 v = *reinterpret_cast<const uint4*>(st + R * 512 + ((q ^ (R & 31)) << 4));
      if (m < a.M && col < F)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v),
                                    reinterpret_cast<u32x4*>(p.keep.gu + m * 2 * F + (q >> 4) * F + col));
    }
    if (a.out == nullptr) return;
    __syncthreads();
  }
  if constexpr (kKeep == kKeep8) {
    // codes as byte rows of 256 columns (128 of G, 128 of U), after the H tile
    char* s8 = st + 256 * 256;
    const int64_t nb = F / 64, blk = k.c0 / 64 + wn;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int R = wm * 128 + 32 * i + r32;
      const int64_t m = k.m0 + R;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t pairs[16], codes[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const f32x16& v = acc[i][2 * w + (t >> 2)];
          const int e = 4 * (t & 3);
          pairs[2 * t] = T::pack2(v[e], v[e + 1]);
          pairs[2 * t + 1] = T::pack2(v[e + 2], v[e + 3]);
        }
        const uint16_t kept = encode_block<T>(pairs, codes);
        if (h == 0 && m < a.M && blk < nb) p.keep.absmax[m * 2 * nb + w * nb + blk] = kept;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const int byte = w * 128 + wn * 64 + 32 * (t >> 2) + 8 * (t & 3) + 4 * h;
          *reinterpret_cast<uint32_t*>(s8 + R * 256 + ((((byte >> 4) ^ R) & 15) << 4) + (byte & 15)) = codes[t];
        }
      }
    }
  }
  // H as 16-bit rows of 128 columns
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int R = wm * 128 + 32 * i + r32;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int q = wn * 8 + 4 * j + jj;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_of<kGelu>(acc[i][j][4 * jj + e]) * acc[i][j + 2][4 * jj + e];
        *reinterpret_cast<uint2*>(st + R * 256 + (((q ^ R) & 15) << 4) + 8 * h) =
            make_uint2(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]));
      }
  }
  __syncthreads();
  const int q = lane & 15;
  const int64_t col = k.c0 + 8 * q;
#pragma unroll 4
  for (int u = 0; u < 16; ++u) {
    const int R = k.wave * 64 + 4 * u + (lane >> 4);
    const int64_t m = k.m0 + R;
    const uint4 v = *reinterpret_cast<const uint4*>(st + R * 256 + (((q ^ R) & 15) << 4));
    if (m < a.M && col < F)
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(a.out + m * F + col));
    if constexpr (kKeep == kKeep8) {
      const uint4 c8 = *reinterpret_cast<const uint4*>(st + 256 * 256 + R * 256 + (((q ^ R) & 15) << 4));
      const int64_t c = k.c0 + 16 * (q & 7);   // chunks 0 .. 7 are G's, 8 .. 15 U's
      if (m < a.M && c < F)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, c8),
                                    reinterpret_cast<u32x4*>(p.keep.codes + m * 2 * F + (q >> 3) * F + c));
    }
  }
}

// The split's fp32 tile: columns c of G at c, of U at F + c of an M x 2F matrix.
template <class Core>
__device__ __forceinline__ void finish_gated_split(const Core& k, const GatedArgs& p, f32x16 (&acc)[4][4]) {
  const BigArgs& a = p.g;
  const int lane = k.lane, r32 = lane & 31, h = lane >> 5, wm = k.wave >> 1, wn = k.wave & 1;
  const int64_t cols = 2 * p.F;
  const Rsrc rp = make_rsrc(a.part + (static_cast<int64_t>(blockIdx.z) * a.M + k.m0) * cols + k.c0,
                            ((a.M - k.m0) * cols - k.c0) * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = wm * 128 + 32 * i + r32;
    const bool row_ok = k.m0 + row < a.M;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int col = wn * 64 + 32 * (j & 1) + 8 * jj + 4 * h;
        const uint32_t voff = (row_ok && k.c0 + col < p.F)
                                  ? static_cast<uint32_t>((row * cols + (j >> 1) * p.F + col) * 4) : kMasked;
        const f32x4 v = {acc[i][j][4 * jj], acc[i][j][4 * jj + 1], acc[i][j][4 * jj + 2], acc[i][j][4 * jj + 3]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rp, voff, 0, 0);
      }
  }
}

// The dense GEMM's loop (dense_loop) with the
// gated epilogue.
template <class T, bool kKTail, bool kSplit, bool kGelu, int kKeep>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void gated_dense_kernel(GatedArgs p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const BigArgs& a = p.g;
  typedef Dense<T, true, kKTail, true> Core;
  Core k(a, smem);
  f32x16 acc[4][4];
  dense_loop<kSplit>(k, a, acc);
  if constexpr (kSplit) finish_gated_split(k, p, acc);
  else finish_gated<T, kGelu, kKeep>(k, p, acc);
}

// After a split GEMM: G and U as the sums of the partials in split order, then
// the epilogue's work.  count: M F / 8 chunks.
template <class T, bool kGelu>
__global__ __launch_bounds__(256) void gated_sum_kernel(const float* __restrict__ part, int64_t splits, int64_t M,
                                                        int64_t F, uint16_t* H, GatedKeep keep) {
  const uint32_t per = static_cast<uint32_t>(F / 8), count = static_cast<uint32_t>(M) * per;
  const int64_t plane = M * 2 * F;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < count; i += gridDim.x * 256) {
    const uint32_t m = i / per;
    const int64_t col = static_cast<int64_t>(i - m * per) * 8;
    f32x4 s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = f32x4{0, 0, 0, 0};
#pragma unroll 4
    for (int64_t z = 0; z < splits; ++z) {
      const float* pg = part + z * plane + m * 2 * F + col;
      s[0] += *reinterpret_cast<const f32x4*>(pg);
      s[1] += *reinterpret_cast<const f32x4*>(pg + 4);
      s[2] += *reinterpret_cast<const f32x4*>(pg + F);
      s[3] += *reinterpret_cast<const f32x4*>(pg + F + 4);
    }
    const float g[8] = {s[0][0], s[0][1], s[0][2], s[0][3], s[1][0], s[1][1], s[1][2], s[1][3]};
    const float u[8] = {s[2][0], s[2][1], s[2][2], s[2][3], s[3][0], s[3][1], s[3][2], s[3][3]};
    gated_store8<T, kGelu>(g, u, m, col, F, H, keep);
  }
}

// dY = [dG | dU] (M x 2F) from dH and the kept G and U.
template <class T, bool kGelu, bool k8>
__global__ __launch_bounds__(256) void gated_dy_kernel(const uint16_t* __restrict__ dH, GatedKeep kept, int64_t M,
                                                       int64_t F, uint16_t* __restrict__ dY) {
  const uint32_t per = static_cast<uint32_t>(F / 8), count = static_cast<uint32_t>(M) * per;
  const int64_t nb = F / 64;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < count; i += gridDim.x * 256) {
    const uint32_t m = i / per;
    const int64_t col = static_cast<int64_t>(i - m * per) * 8;
    const int64_t at = m * 2 * F + col;
    const uint4 d = *reinterpret_cast<const uint4*>(dH + m * F + col);
    uint4 g, u;
    if (k8) {
      const uint2 qg = *reinterpret_cast<const uint2*>(kept.codes + at);
      const uint2 qu = *reinterpret_cast<const uint2*>(kept.codes + at + F);
      const float sg = act8_step<T>(kept.absmax[m * 2 * nb + col / 64]);
      const float su = act8_step<T>(kept.absmax[m * 2 * nb + nb + col / 64]);
      const uint2 g0 = act8_values4<T>(qg.x, sg), g1 = act8_values4<T>(qg.y, sg);
      const uint2 u0 = act8_values4<T>(qu.x, su), u1 = act8_values4<T>(qu.y, su);
      g = make_uint4(g0.x, g0.y, g1.x, g1.y);
      u = make_uint4(u0.x, u0.y, u1.x, u1.y);
    } else {
      g = *reinterpret_cast<const uint4*>(kept.gu + at);
      u = *reinterpret_cast<const uint4*>(kept.gu + at + F);
    }
    const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float vg[2], vu[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int sh = 16 * e;
        float f, df;
        act_grad_of<kGelu>(T::widen((gw[p] >> sh) & 0xffffu), f, df);
        const float dh = T::widen((dw[p] >> sh) & 0xffffu);
        vg[e] = dh * T::widen((uw[p] >> sh) & 0xffffu) * df;
        vu[e] = dh * f;
      }
      og[p] = T::pack2(vg[0], vg[1]);
      ou[p] = T::pack2(vu[0], vu[1]);
    }
    *reinterpret_cast<uint4*>(dY + at) = make_uint4(og[0], og[1], og[2], og[3]);
    *reinterpret_cast<uint4*>(dY + at + F) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

unsigned ew_grid(int64_t chunks) {
  const int64_t b = (chunks + 255) / 256;
  return static_cast<unsigned>(b < 4096 ? b : 4096);
}

template <class T, bool kKTail, bool kSplit, bool kGelu, int kKeep>
hipError_t launch_gated_t(const GatedArgs& p, hipStream_t stream, const Timer& tm) {
  // raised once per process; the initialisation of a function-local static
  // is thread-safe, so concurrent first calls do not race
  static const hipError_t lds_limit =
      hipFuncSetAttribute(reinterpret_cast<const void*>(&gated_dense_kernel<T, kKTail, kSplit, kGelu, kKeep>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, kDenseLds);
  if (lds_limit != hipSuccess) return lds_limit;
  const unsigned zs = kSplit ? static_cast<unsigned>((p.g.K + p.g.k_per - 1) / p.g.k_per) : 1u;
  const dim3 grid(static_cast<unsigned>((p.F + 127) / 128), static_cast<unsigned>((p.g.M + kBM - 1) / kBM), zs);
  hipExtLaunchKernelGGL((gated_dense_kernel<T, kKTail, kSplit, kGelu, kKeep>), grid, dim3(kThreads), kDenseLds, stream,
                        tm.start(), tm.end(), 0, p);
  return hipGetLastError();
}
template <class T, bool kKTail>
hipError_t launch_gated_k(const GatedArgs& p, bool gelu, hipStream_t stream, const Timer& tm) {
  if (p.g.part != nullptr) return launch_gated_t<T, kKTail, true, false, kKeepNone>(p, stream, tm);
  const int keep = p.keep.gu != nullptr ? kKeep16 : (p.keep.codes != nullptr ? kKeep8 : kKeepNone);
  if (gelu) {
    if (keep == kKeep16) return launch_gated_t<T, kKTail, false, true, kKeep16>(p, stream, tm);
    if (keep == kKeep8) return launch_gated_t<T, kKTail, false, true, kKeep8>(p, stream, tm);
    return launch_gated_t<T, kKTail, false, true, kKeepNone>(p, stream, tm);
  }
  if (keep == kKeep16) return launch_gated_t<T, kKTail, false, false, kKeep16>(p, stream, tm);
  if (keep == kKeep8) return launch_gated_t<T, kKTail, false, false, kKeep8>(p, stream, tm);
  return launch_gated_t<T, kKTail, false, false, kKeepNone>(p, stream, tm);
}

}  // namespace

// The GEMM and, after a split one, the sums.  WhatT: 2F x K, Zext: M x 4r, Bt: 2F x r.
hipError_t launch_gated_dense(int64_t M, int64_t K, int64_t F, int64_t r, const uint16_t* X, const uint16_t* WhatT,
                              const uint16_t* Zext, const uint16_t* Bt, bool gelu, uint16_t* H, const GatedKeep& keep,
                              hipStream_t stream, int dtype, void* split_ws) {
  GatedArgs p{};
  p.g = BigArgs{X, K, NF4View{}, Zext, Bt, H, M, K, 2 * F, r, WhatT};
  p.g.ext_a_ld = 4 * r;
  p.keep = keep;
  p.F = F;
  const SplitPlan sp = plan_split(M, 2 * F, K);
  if (sp.splits >= 2) {
    p.g.part = static_cast<float*>(split_ws);
    p.g.k_per = sp.k_per;
  }
  const bool tail = K % kBK != 0;
  hipError_t e;
  {
    const Timer t(QK_GATED_FWD, stream, true);
    if (dtype == kDtypeF16)
      e = tail ? launch_gated_k<F16, true>(p, gelu, stream, t) : launch_gated_k<F16, false>(p, gelu, stream, t);
    else
      e = tail ? launch_gated_k<Bf16, true>(p, gelu, stream, t) : launch_gated_k<Bf16, false>(p, gelu, stream, t);
  }
  if (e != hipSuccess || sp.splits < 2) return e;
  auto* sum = dtype == kDtypeF16 ? (gelu ? gated_sum_kernel<F16, true> : gated_sum_kernel<F16, false>)
                                 : (gelu ? gated_sum_kernel<Bf16, true> : gated_sum_kernel<Bf16, false>);
  Timer tm(QK_REDUCE, stream);
  hipLaunchKernelGGL(sum, dim3(ew_grid(M * F / 8)), dim3(256), 0, stream, p.g.part, sp.splits, M, F, H, keep);
  tm.stop();
  return hipGetLastError();
}

hipError_t launch_gated_dy(int64_t M, int64_t F, const uint16_t* dH, const GatedKeep& kept, bool gelu, uint16_t* dY,
                           hipStream_t stream, int dtype) {
  const bool k8 = kept.codes != nullptr;
  auto pick = [&](auto tag) {
    typedef decltype(tag) T;
    return gelu ? (k8 ? gated_dy_kernel<T, true, true> : gated_dy_kernel<T, true, false>)
                : (k8 ? gated_dy_kernel<T, false, true> : gated_dy_kernel<T, false, false>);
  };
  auto* k = dtype == kDtypeF16 ? pick(F16{}) : pick(Bf16{});
  Timer tm(QK_GATED_DY, stream);
  hipLaunchKernelGGL(k, dim3(ew_grid(M * F / 8)), dim3(256), 0, stream, dH, kept, M, F, dY);
  tm.stop();
  return hipGetLastError();
}

}  // namespace qn
