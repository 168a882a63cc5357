// The gated feed-forward front of the layer for more than 256 rows, on gfx950:
//   [Zg | Zu] = X A,  G = X Ŵg + c Zg Bg,  U = X Ŵu + c Zu Bu,  H = act(G) * U
// and the elementwise half of its backward.  (Up to 256 rows: gemv.hip.)
//
// Forward: one dense GEMM over both weights, dequantized beforehand and stacked
// (2F x K).  A 256 x 256 tile of it takes 128 columns of each weight (kPaired in
// gemm16.hpp), so the lane that holds G of an element also holds its U: the
// activation, the product, the 16-bit rounding and, where the backward wants
// G and U kept in 8 bits, the checkpoint's encoding run on the accumulators,
// and neither G nor U passes through memory to be combined.  Bound by the
// matrix cores and, in several rounds of short tiles, by what lies between them: at
// 4096 x 4096 x 11008 (5.4 rounds of 64 stages, 8 bits kept) 617 to 664 us, the MFMA
// pipes 56 % busy at 2.08 GHz and a CU holding its workgroup 84 % of the launch, where
// dX, one round of 344 stages with the same operations, takes 473 to 509 at 79 %,
// 1.89 GHz and 96 %: tiles' starts and epilogues are bare with one workgroup a CU.
// With few tiles the reduction is split (plan_gated_split) and the fp32 partials
// are summed in split order by gated_sum_kernel, which then does the same.
//
// Backward: dG = dH U act'(G), dU = dH act(G) (gated_dy_kernel, bound by
// memory: 2 bytes of dH, 4 or 2.06 of G and U, 4 written per element), stored
// side by side as the M x 2F gradient of a grouped linear; the rest is that
// linear's backward (layer.hip).  G and U that were not kept are computed
// again by the forward's own kernels.
// dG and dU are rounded to 16 bits there, as every linear's output gradient is: the
// products that read them take 16-bit operands, and fp32 in two parts would double
// both products and the pass.  A training step's outputs are then off by 0.0024 of
// their norm in bf16, 0.0017 with fp32 dG and dU (their own rounding alone).
#include <hip/hip_ext.h>

#include "gated.hpp"
#include "gemm16.hpp"

namespace qn {

namespace {

struct GatedArgs {
  G16Args g;        // act = X, w = [Ŵg | Ŵu]ᵀ (2F x K), ext_a = [hi | lo] of c Z (M x 4r), ext_b = Bᵀ (2F x r)
  GatedKeep keep;
  uint16_t* H;      // null: not wanted (with kKeep16 only)
  int64_t F;
};

enum { kKeepNone = 0, kKeep16 = 1, kKeep8 = 2 };

// The tile's epilogue.  A lane holds, of row 16 i + q and columns wn*64 + 16 j +
// 4 g .. +3, G in acc[i][j] and U in acc[i][j + 4], j < 4.
template <class T, bool kGelu, int kKeep, class Core>
__device__ __forceinline__ void finish_gated(const Core& k, const GatedArgs& p, f32x4 (&acc)[8][8]) {
  const int q = k.q, g = k.g, lane = k.lane;
  const int64_t F = p.F, M = p.g.M;
  char* st = k.smem;
  if constexpr (kKeep == kKeep16) {
    // [G | U]: 16-byte groups 0 .. 15 of a tile row are G's, the others U's
    k.store_rows16(acc, [&](int R, int c, const uint4& v) {
      const int64_t m = k.m0 + R, col = k.c0 + 8 * (c & 15);
      if (m < M && col < F)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v),
                                    reinterpret_cast<u32x4*>(p.keep.gu + m * 2 * F + (c >> 4) * F + col));
    });
    if (p.H == nullptr) return;
    __syncthreads();
  }
  char* s8 = st + 256 * 256;   // codes as byte rows of 256 columns (128 of G, 128 of U), after the H tile
  if constexpr (kKeep == kKeep8) {
    // A block of 64 columns of a row is the wave's 64 of one weight: 16 values in
    // each of the four lanes q, q + 16, q + 32, q + 48.
    const int64_t nb = F / 64, blk = k.c0 / 64 + k.wn;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int R = k.wm * 128 + 16 * i + q;
      const int64_t m = k.m0 + R;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t pair[8], top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4& v = acc[i][4 * w + j];
          pair[2 * j] = T::pack2(v[0], v[1]);
          pair[2 * j + 1] = T::pack2(v[2], v[3]);
          top = act8_max2(top, act8_max2(pair[2 * j] & 0x7fff7fffu, pair[2 * j + 1] & 0x7fff7fffu));
        }
        top = act8_max2(top, __shfl_xor(top, 16, 64));
        top = act8_max2(top, __shfl_xor(top, 32, 64));
        const Act8Scale s = act8_scale<T>(max(top & 0xffffu, top >> 16));
        if (g == 0 && m < M && blk < nb) p.keep.absmax[m * 2 * nb + w * nb + blk] = s.kept;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint32_t*>(s8 + R * 256 + (((w * 8 + k.wn * 4 + j) ^ q) << 4) + 4 * g) =
              act8_codes4<T>(pair[2 * j], pair[2 * j + 1], s);
      }
    }
  }
  // H as 16-bit rows of 128 columns
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int R = k.wm * 128 + 16 * i + q;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_of<kGelu>(acc[i][j][e]) * acc[i][j + 4][e];
      *reinterpret_cast<uint2*>(st + R * 256 + (((k.wn * 8 + 2 * j + (g >> 1)) ^ q) << 4) + 8 * (g & 1)) =
          make_uint2(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]));
    }
  }
  __syncthreads();
  const int c = lane & 15;
  const int64_t col = k.c0 + 8 * c;
#pragma unroll 4
  for (int u = 0; u < 16; ++u) {
    const int R = k.wave * 64 + 4 * u + (lane >> 4);
    const int64_t m = k.m0 + R;
    const uint4 v = *reinterpret_cast<const uint4*>(st + R * 256 + (((c ^ R) & 15) << 4));
    if (m < M && col < F)
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(p.H + m * F + col));
    if constexpr (kKeep == kKeep8) {
      const uint4 c8 = *reinterpret_cast<const uint4*>(s8 + R * 256 + (((c ^ R) & 15) << 4));
      const int64_t at = k.c0 + 16 * (c & 7);   // groups 0 .. 7 are G's, 8 .. 15 U's
      if (m < M && at < F)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, c8),
                                    reinterpret_cast<u32x4*>(p.keep.codes + m * 2 * F + (c >> 3) * F + at));
    }
  }
}

template <class T, bool kSplit, bool kGelu, int kKeep>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void gated_dense_kernel(GatedArgs p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Core16<T, kPaired> k(p.g, smem);
  f32x4 acc[8][8];
  k.template run<kSplit>(acc);
  if constexpr (kSplit) k.store_part(acc, 2 * (p.F - p.g.first));
  else finish_gated<T, kGelu, kKeep>(k, p, acc);
}

// dX = dY Ŵᵀ + dZ Aᵀ.  dZ is 16 bits here: its rounding is as large as dY's beside
// it, which a second part of dZ would leave (dA, which has dZ alone, takes both).
template <class T, bool kSplit>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void gated_dx_kernel(G16Args p,
                                                                                                      uint16_t* dX) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Core16<T, kRows> k(p, smem);
  f32x4 acc[8][8];
  k.template run<kSplit>(acc);
  if constexpr (kSplit) {
    k.store_part(acc, p.wrows);
  } else {
    k.store_rows16(acc, [&](int R, int c, const uint4& v) {
      const int64_t m = k.m0 + R, col = k.c0 + 8 * c;
      if (m < p.M && col < p.wrows)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(dX + m * p.wrows + col));
    });
  }
}

// After a split GEMM of the columns from `first` on: G and U as the sums of the
// partials in split order, then the epilogue's work.
template <class T, bool kGelu>
__global__ __launch_bounds__(256) void gated_sum_kernel(const float* __restrict__ part, int64_t splits, int64_t M,
                                                        int64_t F, int64_t first, uint16_t* H, GatedKeep keep) {
  const int64_t Fs = F - first;
  const uint32_t per = static_cast<uint32_t>(Fs / 8), count = static_cast<uint32_t>(M) * per;
  const int64_t plane = M * 2 * Fs;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < count; i += gridDim.x * 256) {
    const uint32_t m = i / per;
    const int64_t col = static_cast<int64_t>(i - m * per) * 8;
    f32x4 s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = f32x4{0, 0, 0, 0};
#pragma unroll 4
    for (int64_t z = 0; z < splits; ++z) {
      const float* pg = part + z * plane + m * 2 * Fs + col;
      s[0] += *reinterpret_cast<const f32x4*>(pg);
      s[1] += *reinterpret_cast<const f32x4*>(pg + 4);
      s[2] += *reinterpret_cast<const f32x4*>(pg + Fs);
      s[3] += *reinterpret_cast<const f32x4*>(pg + Fs + 4);
    }
    const float g[8] = {s[0][0], s[0][1], s[0][2], s[0][3], s[1][0], s[1][1], s[1][2], s[1][3]};
    const float u[8] = {s[2][0], s[2][1], s[2][2], s[2][3], s[3][0], s[3][1], s[3][2], s[3][3]};
    gated_store8<T, kGelu>(g, u, m, first + col, F, H, keep);
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

template <class T, bool kSplit, bool kGelu, int kKeep>
hipError_t launch_gated_t(const GatedArgs& p, int64_t cols, hipStream_t stream, const Timer& tm) {
  // raised once per process; the initialisation of a function-local static
  // is thread-safe, so concurrent first calls do not race
  static const hipError_t lds_limit =
      hipFuncSetAttribute(reinterpret_cast<const void*>(&gated_dense_kernel<T, kSplit, kGelu, kKeep>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, kG16Lds);
  if (lds_limit != hipSuccess) return lds_limit;
  const unsigned zs = kSplit ? static_cast<unsigned>((p.g.red + p.g.k_per - 1) / p.g.k_per) : 1u;
  const dim3 grid(static_cast<unsigned>((cols + 127) / 128), static_cast<unsigned>((p.g.M + kBM - 1) / kBM), zs);
  hipExtLaunchKernelGGL((gated_dense_kernel<T, kSplit, kGelu, kKeep>), grid, dim3(kThreads), kG16Lds, stream, tm.start(),
                        tm.end(), 0, p);
  return hipGetLastError();
}
template <class T>
hipError_t launch_gated_k(const GatedArgs& p, int64_t cols, bool gelu, hipStream_t stream, const Timer& tm) {
  if (p.g.part != nullptr) return launch_gated_t<T, true, false, kKeepNone>(p, cols, stream, tm);
  const int keep = p.keep.gu != nullptr ? kKeep16 : (p.keep.codes != nullptr ? kKeep8 : kKeepNone);
  if (gelu) {
    if (keep == kKeep16) return launch_gated_t<T, false, true, kKeep16>(p, cols, stream, tm);
    if (keep == kKeep8) return launch_gated_t<T, false, true, kKeep8>(p, cols, stream, tm);
    return launch_gated_t<T, false, true, kKeepNone>(p, cols, stream, tm);
  }
  if (keep == kKeep16) return launch_gated_t<T, false, false, kKeep16>(p, cols, stream, tm);
  if (keep == kKeep8) return launch_gated_t<T, false, false, kKeep8>(p, cols, stream, tm);
  return launch_gated_t<T, false, false, kKeepNone>(p, cols, stream, tm);
}
template <class T, bool kSplit>
hipError_t launch_gated_dx_t(const G16Args& p, uint16_t* dX, hipStream_t stream, const Timer& tm) {
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&gated_dx_kernel<T, kSplit>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, kG16Lds);
  if (lds_limit != hipSuccess) return lds_limit;
  const unsigned zs = kSplit ? static_cast<unsigned>((p.red + p.k_per - 1) / p.k_per) : 1u;
  const dim3 grid(static_cast<unsigned>((p.wrows + kBN - 1) / kBN), static_cast<unsigned>((p.M + kBM - 1) / kBM), zs);
  hipExtLaunchKernelGGL((gated_dx_kernel<T, kSplit>), grid, dim3(kThreads), kG16Lds, stream, tm.start(), tm.end(), 0, p, dX);
  return hipGetLastError();
}

}  // namespace

// The split of a Core16 product of M x cols outputs: the one of least estimated
// time, where a CU takes kStageUs for a 64-element stage and kTileUs besides them
// for a tile, tiles run in rounds of 256, and partials go through memory twice at
// kBytesPerUs, added by one more launch.  (The dense kernels' plan_split fills the
// device at most once and bounds the partials to 32 MiB: it left dX of 770 rows,
// K 5568, F 19520, 88 tiles of 610 stages, whole, 705 us; with this plan, and the
// forward's, that training step takes 1490 us instead of 1857.)
SplitPlan plan_split16(int64_t M, int64_t cols, int64_t red) {
  constexpr double kStageUs = 1.4, kTileUs = 5.0, kBytesPerUs = 5e6, kLaunchUs = 4.0, kAddUs = 0.1;
  // (32-bit: a call's host time goes into these divisions)
  const uint32_t tiles = static_cast<uint32_t>(((M + kBM - 1) / kBM) * ((cols + kBN - 1) / kBN));
  const uint32_t stages = static_cast<uint32_t>((red + kBK - 1) / kBK);
  const int64_t plane = M * cols * 4;
  SplitPlan best{1, red, 0};
  if (tiles >= 256) return best;
  double least = kStageUs * stages + kTileUs;
  for (uint32_t s = 2; 4 * s <= stages && s <= 64 && s * tiles <= 1024; ++s) {
    const uint32_t per = (stages + s - 1) / s, splits = (stages + per - 1) / per;
    if (splits * plane > (int64_t(1) << 28)) break;
    const double us = ((tiles * splits + 255) / 256) * (kStageUs * per + kTileUs) +
                      static_cast<double>(splits * plane) * (2.0 / kBytesPerUs) + kLaunchUs + kAddUs * splits;
    if (us >= least) continue;
    least = us;
    best = SplitPlan{splits, static_cast<int64_t>(per) * kBK, (splits * plane + 255) / 256 * 256};
  }
  return best;
}

// Fewer than 256 tiles: plan_split16's, of all columns (first = 0).  More: the
// tiles run in rounds of 256, one a CU, and a last round of few leaves most CUs
// idle; there the column tiles past the full rounds are split alone, where the
// estimate (as plan_split16's) says so.  After two full rounds it does not pay:
// the others then run at the power limit, and what idle CUs leave goes to them.
// Whole forward product, split and not: 375 rows, K 7064, F 19072 (298 tiles)
// 256 and 350 us; 4096 rows, K 4096, F 11008 (1376 tiles, 5 rounds and 96) 657 and
// 651; 2048 rows, K 8192, F 22016 (as many) 1168 and 1157.
GatedSplit plan_gated_split(int64_t M, int64_t K, int64_t F) {
  constexpr int64_t kTailRounds = 2;
  const int64_t mt = (M + kBM - 1) / kBM, nt = (F + 127) / 128;
  const int64_t full = mt * nt / 256, n1 = full * 256 / mt;   // column tiles of the full rounds
  if (full > kTailRounds || n1 >= nt) return GatedSplit{F, 1, K, 0};
  const SplitPlan sp = plan_split16(M, 2 * (F - 128 * n1), K);
  if (sp.splits < 2) return GatedSplit{F, 1, K, 0};
  return GatedSplit{128 * n1, sp.splits, sp.k_per, sp.part_bytes};
}

// The GEMM and, after a split one, the sums.  WhatT: 2F x K, Zext: M x 4r, Bt: 2F x r.
hipError_t launch_gated_dense(int64_t M, int64_t K, int64_t F, int64_t r, const uint16_t* X, const uint16_t* WhatT,
                              int64_t w_ld, const uint16_t* Zext, const uint16_t* Bt, bool gelu, uint16_t* H, const GatedKeep& keep,
                              hipStream_t stream, int dtype, void* split_ws) {
  GatedArgs p{};
  p.g = G16Args{X, K, WhatT, w_ld, M, 2 * F, K, Zext, 4 * r, Bt, r, nullptr, 0};
  p.keep = keep;
  p.H = H;
  p.F = F;
  const GatedSplit sp = plan_gated_split(M, K, F);
  hipError_t e = hipSuccess;
  if (sp.first > 0) {
    const Timer t(QK_GATED_FWD, stream, true);
    e = dtype == kDtypeF16 ? launch_gated_k<F16>(p, sp.first, gelu, stream, t) : launch_gated_k<Bf16>(p, sp.first, gelu, stream, t);
  }
  if (e != hipSuccess || sp.splits < 2) return e;
  p.g.part = static_cast<float*>(split_ws);
  p.g.k_per = sp.k_per;
  p.g.first = sp.first;
  {
    const Timer t(QK_GATED_FWD, stream, true);
    e = dtype == kDtypeF16 ? launch_gated_k<F16>(p, F - sp.first, gelu, stream, t)
                           : launch_gated_k<Bf16>(p, F - sp.first, gelu, stream, t);
  }
  if (e != hipSuccess) return e;
  auto* sum = dtype == kDtypeF16 ? (gelu ? gated_sum_kernel<F16, true> : gated_sum_kernel<F16, false>)
                                 : (gelu ? gated_sum_kernel<Bf16, true> : gated_sum_kernel<Bf16, false>);
  Timer tm(QK_REDUCE, stream);
  hipLaunchKernelGGL(sum, dim3(ew_grid(M * (F - sp.first) / 8)), dim3(256), 0, stream, p.g.part, sp.splits, M, F, sp.first,
                     H, keep);
  tm.stop();
  return hipGetLastError();
}

hipError_t launch_gated_dx(int64_t M, int64_t K, int64_t red, int64_t rt, const uint16_t* dY, const uint16_t* What,
                           const uint16_t* dZ, const uint16_t* A, uint16_t* dX, hipStream_t stream, int dtype,
                           void* split_ws) {
  G16Args p{dY, red, What, red, M, K, red, dZ, rt, A, rt, nullptr, 0};
  const SplitPlan sp = plan_split16(M, K, red);
  if (sp.splits >= 2) {
    p.part = static_cast<float*>(split_ws);
    p.k_per = sp.k_per;
  }
  hipError_t e;
  {
    const Timer t(QK_BWD_DX, stream, true);
    if (dtype == kDtypeF16)
      e = p.part != nullptr ? launch_gated_dx_t<F16, true>(p, dX, stream, t) : launch_gated_dx_t<F16, false>(p, dX, stream, t);
    else
      e = p.part != nullptr ? launch_gated_dx_t<Bf16, true>(p, dX, stream, t) : launch_gated_dx_t<Bf16, false>(p, dX, stream, t);
  }
  if (e != hipSuccess || sp.splits < 2) return e;
  return launch_split_sum(p.part, sp.splits, M * K, dX, stream, dtype);
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
