// Large-M GEMM kernels for gfx950: the forward Y = X Ŵ + c Z B and the
// backward dX = G Ŵᵀ + dZ Aᵀ (page "QLoRA：冻结的 4-bit 权重怎样参与一次微调",
// sections "量化基座与可训练支路怎样相加" and "冻结权重为什么仍然需要输入梯度").
//
// Both kernels: workgroup of 256 threads (4 waves, 2 x 2), output tile
// 256 x 256, each wave 128 x 128 as 4 x 4 tiles of v_mfma_f32_32x32x16_bf16
// (256 fp32 accumulators per lane in AGPRs, one wave per SIMD).  The LoRA
// term is r more reduction steps over (Z, (c B)ᵀ) or (dZ, A) after the main
// loop; the bf16 tile is then stored through LDS as whole rows.
//
// qlora_big_kernel (17 <= M < 192) decodes the packed weight inside its
// reduction loop.  Per 64-element stage the workgroup
//   - copies the activation tile of stage s+1 from global memory straight into
//     LDS (buffer loads with the LDS destination, no registers involved);
//   - loads the code words and block scales of stage s+2 into registers;
//   - builds the bf16 block tables of stage s+1 (16 entries RNE(fl32(C[j]*â))
//     per 64-weight block row) and decodes stage s+1 into the other weight
//     buffer by table lookups (no per-weight multiply or conversion);
//   - runs the 64 MFMAs of stage s;
// then waits for its loads and synchronises once.  LDS layout of one operand
// stage: 256 rows x 64 bf16 (128 bytes per row), the eight 16-byte chunks of
// row r stored at chunk ^ ((r ^ r >> 3) & 7), which keeps the fragment reads
// and the decoder's writes free of bank conflicts per 8 lanes.
//  - forward weight (reduction over k, codes packed along n): thread (rg, cg)
//    owns k-rows 8rg..8rg+7 and columns 8cg..8cg+7 of the stage; it builds the
//    table of one (row, block) pair that the 8 threads of its group share
//    and writes each column's 8 k-values as one chunk;
//  - backward weight (reduction over n, the packed direction): thread t owns
//    k-row t and the stage's 64 n, exactly one block and one table.
// Rows at or past K get an all-zero table and the matching activation
// chunks are masked, so tails add exact zeros.
//
// qlora_dense_kernel (M >= 192) reads a weight dequantized beforehand to bf16
// (bit-identical to the fused decode) and streams 64-element stages through three
// LDS slots of activations and two of weights, whole cache lines per copy (see Dense).
//
// Every global load is a raw buffer load, so masked lanes need no branches:
// a lane whose row, column or reduction index lies outside its operand
// (tails, and the prefetches that run past the last stage) gets a per-lane
// offset past the buffer's size, whatever the scalar stage offset added.
// The MFMA is issued as D = Ŵ-fragment x activation-fragment, so each lane
// holds 4 consecutive output columns of one output row.
#include <hip/hip_ext.h>

#include "gemm_core.hpp"

namespace qn {

namespace {

template <class T, bool kForward, bool kKTail, bool kSplit>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void qlora_big_kernel(BigArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Big<T, kForward, kKTail> k(a, smem);
  {
    float* q2t = reinterpret_cast<float*>(smem + kOffQ);
    q2t[k.t] = q2_value(k.t - 128);
  }
  int64_t s_beg, s_end;
  stage_range<kSplit>(a, k.red, kBK, s_beg, s_end);

  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // prologue: the first stage into buffer 0, the next one's weights into registers
  WRegs cur, nxt;
  k.copy_act(s_beg, 0);
  k.load_w(cur, s_beg);
  k.load_w(nxt, s_beg + 1);
  __syncthreads();                 // q2t staged
  k.build_table(cur, s_beg, 0);
  {
    uint32_t ix[16];
    k.split_codes(cur, ix);
#pragma unroll
    for (int p = 0; p < 8; ++p) k.decode_part(ix, 0, p);
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  cur = nxt;

  for (int64_t s = s_beg; s < s_end; ++s) {
    const int b = static_cast<int>((s - s_beg) & 1);
    // (stage s+1 and s+2 accesses past the range are masked or never read)
    k.copy_act(s + 1, b ^ 1);
    k.load_w(nxt, s + 2);
    k.build_table(cur, s + 1, b ^ 1);
    uint32_t ix[16];
    k.split_codes(cur, ix);
    // MFMAs of stage s, with the fragments of substep ks+1 and two decode
    // parts of stage s+1 issued in the shadow of substep ks.
    typename Big<T, kForward, kKTail>::Frags F0, F1;
    k.load_frags(b, 0, F0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks < 3) k.load_frags(b, ks + 1, F1);
      k.decode_part(ix, b ^ 1, 2 * ks);
      k.decode_part(ix, b ^ 1, 2 * ks + 1);
      Big<T, kForward, kKTail>::mma(F0, acc);
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);   // VALU
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // DS read
      }
      __builtin_amdgcn_sched_group_barrier(0x200, 2, 0);     // DS write
      if (ks < 3) F0 = F1;
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    cur = nxt;
  }

  finish<T, kForward, kSplit, true>(k, a, acc);
}

template <class T, bool kForward, bool kKTail, bool kSplit>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void qlora_dense_kernel(BigArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Dense<T, kForward, kKTail> k(a, smem);
  f32x16 acc[4][4];
  dense_loop<kSplit>(k, a, acc);
  finish<T, kForward, kSplit, false>(k, a, acc);
}

template <class T, bool kForward, bool kKTail, bool kSplit>
hipError_t launch_big_t(const BigArgs& a, hipStream_t stream, const Timer& tm) {
  // raised once per process; the initialisation of a function-local static
  // is thread-safe, so concurrent first calls do not race
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&qlora_big_kernel<T, kForward, kKTail, kSplit>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes);
  if (lds_limit != hipSuccess) return lds_limit;
  const int64_t cols = kForward ? a.N : a.K, red = kForward ? a.K : a.N;
  const unsigned zs = kSplit ? static_cast<unsigned>((red + a.k_per - 1) / a.k_per) : 1u;
  dim3 grid(static_cast<unsigned>((cols + kBN - 1) / kBN), static_cast<unsigned>((a.M + kBM - 1) / kBM), zs);
  hipExtLaunchKernelGGL((qlora_big_kernel<T, kForward, kKTail, kSplit>), grid, dim3(kThreads), kLdsBytes, stream,
                        tm.start(), tm.end(), 0, a);
  return hipGetLastError();
}

template <class T, bool kForward, bool kKTail, bool kSplit>
hipError_t launch_dense_t(const BigArgs& a, hipStream_t stream, const Timer& tm) {
  // raised once per process; the initialisation of a function-local static
  // is thread-safe, so concurrent first calls do not race
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&qlora_dense_kernel<T, kForward, kKTail, kSplit>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, kDenseLds);
  if (lds_limit != hipSuccess) return lds_limit;
  const int64_t cols = kForward ? a.N : a.K, red = kForward ? a.K : a.N;
  const unsigned zs = kSplit ? static_cast<unsigned>((red + a.k_per - 1) / a.k_per) : 1u;
  dim3 grid(static_cast<unsigned>((cols + kBN - 1) / kBN), static_cast<unsigned>((a.M + kBM - 1) / kBM), zs);
  hipExtLaunchKernelGGL((qlora_dense_kernel<T, kForward, kKTail, kSplit>), grid, dim3(kThreads), kDenseLds, stream,
                        tm.start(), tm.end(), 0, a);
  return hipGetLastError();
}

// Instantiation by compute type, reduction tail and split.
template <bool kForward, bool kDense, class T, bool kKTail>
hipError_t launch_gemm_s(const BigArgs& a, hipStream_t stream, const Timer& tm) {
  if (kDense)
    return a.part != nullptr ? launch_dense_t<T, kForward, kKTail, true>(a, stream, tm)
                             : launch_dense_t<T, kForward, kKTail, false>(a, stream, tm);
  return a.part != nullptr ? launch_big_t<T, kForward, kKTail, true>(a, stream, tm)
                           : launch_big_t<T, kForward, kKTail, false>(a, stream, tm);
}
template <bool kForward, bool kDense, class T>
hipError_t launch_gemm_t(const BigArgs& a, hipStream_t stream, const Timer& tm) {
  const int64_t red = kForward ? a.K : a.N;
  return (red % kBK) ? launch_gemm_s<kForward, kDense, T, true>(a, stream, tm)
                     : launch_gemm_s<kForward, kDense, T, false>(a, stream, tm);
}
template <bool kForward, bool kDense>
hipError_t launch_gemm(const BigArgs& a, hipStream_t stream, const Timer& tm, int dtype) {
  return dtype == F16::kDtype ? launch_gemm_t<kForward, kDense, F16>(a, stream, tm)
                              : launch_gemm_t<kForward, kDense, Bf16>(a, stream, tm);
}

// out = the 16-bit rounding of sum_z part[z] (z in order, fp32), 8 elements
// per thread and step; count % 8 == 0.
template <class T>
__global__ __launch_bounds__(256) void split_sum_kernel(const float* __restrict__ part, int64_t splits, int64_t count,
                                                        uint16_t* __restrict__ out) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256 * 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8; i < count; i += stride) {
    f32x4 lo = *reinterpret_cast<const f32x4*>(part + i);
    f32x4 hi = *reinterpret_cast<const f32x4*>(part + i + 4);
#pragma unroll 4
    for (int64_t z = 1; z < splits; ++z) {
      const float* p = part + z * count + i;
      lo += *reinterpret_cast<const f32x4*>(p);
      hi += *reinterpret_cast<const f32x4*>(p + 4);
    }
    *reinterpret_cast<uint4*>(out + i) =
        make_uint4(T::pack2(lo[0], lo[1]), T::pack2(lo[2], lo[3]), T::pack2(hi[0], hi[1]), T::pack2(hi[2], hi[3]));
  }
}

// Attach the split plan of an M x cols output over a reduction of red to a
// (part_ws null: no split).
void attach_split(BigArgs& a, int64_t cols, int64_t red, void* part_ws) {
  const SplitPlan sp = plan_split(a.M, cols, red);
  if (part_ws == nullptr || sp.splits < 2) return;
  a.part = static_cast<float*>(part_ws);
  a.k_per = sp.k_per;
}

// After a split GEMM: the fixed-order sum into the 16-bit output.
hipError_t split_sum(const BigArgs& a, int64_t cols, hipStream_t stream, int dtype) {
  if (a.part == nullptr) return hipGetLastError();
  const int64_t red = cols == a.N ? a.K : a.N;
  return launch_split_sum(a.part, (red + a.k_per - 1) / a.k_per, a.M * cols, a.out, stream, dtype);
}

#ifndef QN_SPLIT_TARGET
#define QN_SPLIT_TARGET 256
#endif
#ifndef QN_SPLIT_MIN_STAGES
#define QN_SPLIT_MIN_STAGES 4
#endif
#ifndef QN_SPLIT_BUDGET_MB
#define QN_SPLIT_BUDGET_MB 32
#endif

}  // namespace

// One 256 x 256 tile per workgroup and one workgroup per CU: with fewer
// tiles than about 256 the reduction is split so that splits x tiles stays
// within 256 workgroups, each split at least QN_SPLIT_MIN_STAGES 64-element
// stages long, and the fp32 partials (written once, read once) within
// QN_SPLIT_BUDGET_MB: past that their traffic costs more than the idle CUs.
SplitPlan plan_split(int64_t M, int64_t cols, int64_t red) {
  const int64_t tiles = ((M + kBM - 1) / kBM) * ((cols + kBN - 1) / kBN);
  int64_t s = QN_SPLIT_TARGET / tiles;
  const int64_t max_s = red / (kBK * QN_SPLIT_MIN_STAGES);
  const int64_t budget_s = (static_cast<int64_t>(QN_SPLIT_BUDGET_MB) << 20) / (M * cols * 4);
  if (s > max_s) s = max_s;
  if (s > budget_s) s = budget_s;
  if (s < 2) return SplitPlan{1, red, 0};
  const int64_t per = ((red + s - 1) / s + kBK - 1) / kBK * kBK;
  const int64_t splits = (red + per - 1) / per;
  if (splits < 2) return SplitPlan{1, red, 0};
  return SplitPlan{splits, per, (splits * M * cols * 4 + 255) / 256 * 256};
}

hipError_t launch_split_sum(const float* part, int64_t splits, int64_t count, uint16_t* out, hipStream_t stream,
                            int dtype) {
  int64_t blocks = (count / 8 + 255) / 256;
  if (blocks > 4096) blocks = 4096;
  Timer tm(QK_REDUCE, stream);
  if (dtype == F16::kDtype)
    hipLaunchKernelGGL(split_sum_kernel<F16>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, part, splits,
                       count, out);
  else
    hipLaunchKernelGGL(split_sum_kernel<Bf16>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, part, splits,
                       count, out);
  tm.stop();
  return hipGetLastError();
}

hipError_t launch_fwd_dense(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, const uint16_t* WhatT,
                            const uint16_t* Z, const uint16_t* cBt, uint16_t* Y, hipStream_t stream, int dtype,
                            void* split_ws) {
  BigArgs a{X, K, NF4View{}, Z, cBt, Y, M, K, N, r, WhatT};
  attach_split(a, N, K, split_ws);
  hipError_t e;
  {
    const Timer t(QK_FWD_GEMM, stream, true);
    if ((e = launch_gemm<true, true>(a, stream, t, dtype)) != hipSuccess) return e;
  }
  return split_sum(a, N, stream, dtype);
}

hipError_t launch_fwd_dense_grouped(int64_t M, int64_t K, int64_t Ntot, int64_t r, const uint16_t* X,
                                    const uint16_t* WhatT, const uint16_t* Zcat, int g, const int64_t* gend,
                                    const uint16_t* cBt, uint16_t* Y, hipStream_t stream, int dtype, void* split_ws) {
  BigArgs a{X, K, NF4View{}, Zcat, cBt, Y, M, K, Ntot, r, WhatT};
  a.ext_a_ld = g * r;
  a.ngroups = g - 1;
  for (int i = 0; i + 1 < g; ++i) a.gend[i] = gend[i];
  attach_split(a, Ntot, K, split_ws);
  hipError_t e;
  {
    const Timer t(QK_FWD_GEMM, stream, true);
    if ((e = launch_gemm<true, true>(a, stream, t, dtype)) != hipSuccess) return e;
  }
  return split_sum(a, Ntot, stream, dtype);
}

hipError_t launch_dx_dense(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, const uint16_t* What,
                           const uint16_t* dZ, const uint16_t* A, uint16_t* dX, hipStream_t stream, int dtype,
                           void* split_ws) {
  BigArgs a{G, N, NF4View{}, dZ, A, dX, M, K, N, r, What};
  attach_split(a, K, N, split_ws);
  hipError_t e;
  {
    const Timer t(QK_BWD_DX, stream, true);
    if ((e = launch_gemm<false, true>(a, stream, t, dtype)) != hipSuccess) return e;
  }
  return split_sum(a, K, stream, dtype);
}

hipError_t launch_fwd_big(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, NF4View W,
                          const uint16_t* Z, const uint16_t* cBt, uint16_t* Y, hipStream_t stream, int dtype,
                          void* split_ws) {
  BigArgs a{X, K, W, Z, cBt, Y, M, K, N, r, nullptr};
  attach_split(a, N, K, split_ws);
  hipError_t e;
  {
    const Timer t(QK_FWD_GEMM, stream, true);
    if ((e = launch_gemm<true, false>(a, stream, t, dtype)) != hipSuccess) return e;
  }
  return split_sum(a, N, stream, dtype);
}

hipError_t launch_dx_big(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, NF4View W,
                         const uint16_t* dZ, const uint16_t* A, uint16_t* dX, hipStream_t stream, int dtype,
                         void* split_ws) {
  BigArgs a{G, N, W, dZ, A, dX, M, K, N, r, nullptr};
  attach_split(a, K, N, split_ws);
  hipError_t e;
  {
    const Timer t(QK_BWD_DX, stream, true);
    if ((e = launch_gemm<false, false>(a, stream, t, dtype)) != hipSuccess) return e;
  }
  return split_sum(a, K, stream, dtype);
}

}  // namespace qn
