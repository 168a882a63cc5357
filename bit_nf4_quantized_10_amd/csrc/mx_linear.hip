// Products of MXFP4 matrices for gfx950 and the layer on such a weight:
//   C = P Qᵀ (both held in MXFP4),
//   Y = Q(X) Wᵀ + c Z B, Z = X A, and its backward.
// Every product runs on v_mfma_scale_f32_16x16x128_f8f6f4, whose operand is a lane's
// block of 32 elements with its scale (mxfp4.hpp): nothing is decoded.
//
// Direct kernel: a wave computes 64 x 64 outputs with both operands loaded from memory
// into its fragments, four steps of 128 elements (one word of scales a row) at a time.
#include <hip/hip_ext.h>

#include "common.hpp"
#include "kernels.hpp"
#include "mx_core.hpp"
#include "mxfp4.hpp"

namespace qn {

namespace {

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
template <class T>
__global__ __launch_bounds__(256) void mx_direct_kernel(MxProductArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane & 15, g = lane >> 4;
  const int64_t M = p.act.rows, N = p.w.rows, K = p.act.cols;
  const int64_t nb = mx_blocks(K), chunks = mx_chunks(K);
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * 64, m0 = static_cast<int64_t>(blockIdx.y) * 64;
  if (n0 >= N) return;
  const Rsrc ra = make_rsrc(p.act.codes, M * nb * 16), rw = make_rsrc(p.w.codes, N * nb * 16);
  const Rsrc rsa = make_rsrc(p.act.scales, mx_scale_bytes(M, K)), rsw = make_rsrc(p.w.scales, mx_scale_bytes(N, K));
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const int64_t c0 = static_cast<int64_t>(blockIdx.z) * p.chunks_per;
  const int64_t c1 = c0 + p.chunks_per < chunks ? c0 + p.chunks_per : chunks;
  for (int64_t c = c0; c < c1; ++c) {
    uint32_t sa[4], sw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // tiles past the last one are past the buffer's end: zeros
      sa[i] = ld_b32(rsa, static_cast<uint32_t>(((m0 / 16 + i) * chunks + c) * 256 + 4 * lane));
      sw[i] = ld_b32(rsw, static_cast<uint32_t>(((n0 / 16 + i) * chunks + c) * 256 + 4 * lane));
    }
    auto step = [&](auto tag) {
      constexpr int s = decltype(tag)::value;
      const int64_t b = c * 16 + 4 * s + g;
      i32x4 fa[4], fw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 16 * i + q, n = n0 + 16 * i + q;
        fa[i] = __builtin_bit_cast(i32x4, ld_b128(ra, m < M && b < nb ? static_cast<uint32_t>((m * nb + b) * 16) : kMasked));
        fw[i] = __builtin_bit_cast(i32x4, ld_b128(rw, n < N && b < nb ? static_cast<uint32_t>((n * nb + b) * 16) : kMasked));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma_mx<s>(fw[j], fa[i], acc[i][j], sw[j], sa[i]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }
  if (blockIdx.z == 0 && p.r > 0) {
    const Rsrc re = make_rsrc(p.ext_a, M * p.r * 2), rb = make_rsrc(p.ext_b, N * p.r * 2);
    for (int64_t j0 = 0; j0 < p.r; j0 += 32) {
      const int64_t e = j0 + 8 * g;
      typename T::v8 fa[4], fw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 16 * i + q, n = n0 + 16 * i + q;
        fa[i] = __builtin_bit_cast(typename T::v8, ld_b128(re, m < M && e < p.r ? static_cast<uint32_t>((m * p.r + e) * 2) : kMasked));
        fw[i] = __builtin_bit_cast(typename T::v8, ld_b128(rb, n < N && e < p.r ? static_cast<uint32_t>((n * p.r + e) * 2) : kMasked));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = T::mfma16(fw[j], fa[i], acc[i][j]);
    }
  }
  float* out = static_cast<float*>(p.out) + static_cast<int64_t>(blockIdx.z) * M * N;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + 16 * i + q;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + 16 * j + 4 * g;
      if (m < M && n < N) *reinterpret_cast<f32x4*>(out + m * N + n) = acc[i][j];
    }
  }
}

template <class T, bool k32>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void mx_tile_kernel(MxProductArgs p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  CoreMx<T> k(p, smem);
  f32x16 acc[4][4];
  k.run(acc);
  if constexpr (k32) k.store32(acc);
  else k.store16(acc);
}

// out = the sum of the splits' fp32 planes in order, in the output's type.
__global__ __launch_bounds__(256) void mx_sum32_kernel(const float* __restrict__ part, int64_t splits, int64_t count,
                                                       float* __restrict__ out) {
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < count; i += static_cast<int64_t>(gridDim.x) * 1024) {
    f32x4 s = *reinterpret_cast<const f32x4*>(part + i);
    for (int64_t z = 1; z < splits; ++z) s += *reinterpret_cast<const f32x4*>(part + z * count + i);
    *reinterpret_cast<f32x4*>(out + i) = s;
  }
}

// How a product runs: by the direct kernel or by tiles, in how many splits of the
// reduction (by chunks); part_bytes: the splits' fp32 planes.
struct MxPlan {
  bool tiles;
  int64_t splits, chunks_per, part_bytes;
};
#ifndef QN_MX_DIRECT_M
#define QN_MX_DIRECT_M 64
#endif
#ifndef QN_MX_STAGE_US
#define QN_MX_STAGE_US 1.2
#endif
MxPlan plan_mx(int64_t M, int64_t N, int64_t K) {
  const int64_t chunks = mx_chunks(K);
  MxPlan pl{M > QN_MX_DIRECT_M, 1, chunks, 0};
  if (!pl.tiles) {
    const int64_t wgs = cdiv(M, 64) * cdiv(N, 256);
    int64_t s = cdiv(512, wgs);
    s = s > chunks ? chunks : s;
    pl.chunks_per = cdiv(chunks, s);
    pl.splits = cdiv(chunks, pl.chunks_per);
    pl.part_bytes = align256(pl.splits * M * N * 4);
    return pl;
  }
  // the split of least estimated time, as plan_split16's: rounds of 256 tiles, the
  // partials through memory twice and one more launch
  constexpr double kStageUs = QN_MX_STAGE_US, kTileUs = 5.0, kBytesPerUs = 5e6, kLaunchUs = 4.0;
  const int64_t tiles = cdiv(M, 256) * cdiv(N, 256), plane = M * N * 4;
  double least = 2 * kStageUs * chunks + kTileUs;
  if (tiles >= 256) return pl;
  for (int64_t s = 2; s <= chunks && s <= 64 && s * tiles <= 1024; ++s) {
    const int64_t per = cdiv(chunks, s), splits = cdiv(chunks, per);
    if (splits * plane > (int64_t(1) << 28)) break;
    const double us = cdiv(tiles * splits, 256) * (2 * kStageUs * per + kTileUs) + static_cast<double>(splits * plane) * (2.0 / kBytesPerUs) +
                      kLaunchUs + 0.1 * splits;
    if (us >= least) continue;
    least = us;
    pl.splits = splits;
    pl.chunks_per = per;
    pl.part_bytes = align256(splits * plane);
  }
  return pl;
}

template <class T, bool k32>
hipError_t launch_mx_tiles_t(const MxProductArgs& p, int64_t splits, hipStream_t stream, const Timer& tm) {
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&mx_tile_kernel<T, k32>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, kG16Lds);
  if (lds_limit != hipSuccess) return lds_limit;
  const dim3 grid(static_cast<unsigned>(cdiv(p.w.rows, 256)), static_cast<unsigned>(cdiv(p.act.rows, 256)), static_cast<unsigned>(splits));
  hipExtLaunchKernelGGL((mx_tile_kernel<T, k32>), grid, dim3(kThreads), kG16Lds, stream, tm.start(), tm.end(), 0, p);
  return hipGetLastError();
}

// out_type: NF4_OUT_*; the adapter's operands are of the 16-bit type dtype.
hipError_t mx_product(MxView act, MxView w, const uint16_t* ext_a, const uint16_t* ext_b, int64_t r, int dtype,
                      int out_type, void* out, void* ws, hipStream_t stream) {
  const int64_t M = act.rows, N = w.rows;
  const MxPlan pl = plan_mx(M, N, act.cols);
  const bool parts = !pl.tiles || pl.splits > 1;
  MxProductArgs p{act, w, ext_a, ext_b, r, parts ? ws : out, pl.chunks_per};
  hipError_t e;
  {
    const Timer tm(QK_MX_GEMM, stream, true);
    if (pl.tiles) {
      const bool k32 = parts || out_type == NF4_OUT_F32;
      if (dtype == kDtypeF16) e = k32 ? launch_mx_tiles_t<F16, true>(p, pl.splits, stream, tm) : launch_mx_tiles_t<F16, false>(p, pl.splits, stream, tm);
      else e = k32 ? launch_mx_tiles_t<Bf16, true>(p, pl.splits, stream, tm) : launch_mx_tiles_t<Bf16, false>(p, pl.splits, stream, tm);
    } else {
      const dim3 grid(static_cast<unsigned>(cdiv(N, 256)), static_cast<unsigned>(cdiv(M, 64)), static_cast<unsigned>(pl.splits));
      hipExtLaunchKernelGGL((dtype == kDtypeF16 ? mx_direct_kernel<F16> : mx_direct_kernel<Bf16>), grid, dim3(256), 0, stream,
                            tm.start(), tm.end(), 0, p);
      e = hipGetLastError();
    }
  }
  if (e != hipSuccess || !parts) return e;
  const float* part = static_cast<const float*>(ws);
  if (out_type != NF4_OUT_F32)
    return launch_split_sum(part, pl.splits, M * N, static_cast<uint16_t*>(out), stream,
                            out_type == NF4_OUT_F16 ? kDtypeF16 : kDtypeBf16);
  const int64_t blocks = cdiv(M * N, 1024);
  Timer tm(QK_REDUCE, stream);
  hipLaunchKernelGGL(mx_sum32_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, part,
                     pl.splits, M * N, static_cast<float*>(out));
  tm.stop();
  return hipGetLastError();
}

}  // namespace

int64_t mx_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) { return plan_mx(M, N, K).part_bytes; }

hipError_t launch_mx_matmul(MxView p, MxView q, int out_type, void* out, void* ws, hipStream_t stream) {
  return mx_product(p, q, nullptr, nullptr, 0, out_type == NF4_OUT_F16 ? kDtypeF16 : kDtypeBf16, out_type, out, ws, stream);
}

// Workspace of the forward: Aᵀ, Z's partials, (c B)ᵀ, X's codes and scales, the
// product's partials, Z for calls that do not pass it.
int64_t mx_fwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t r) {
  const SkinnyPlan p = plan_skinny(M, K, N, r);
  return p.at_bytes + p.z_part + align256(N * r * 2) + align256(mx_code_bytes(M, K)) + align256(mx_scale_bytes(M, K)) +
         plan_mx(M, N, K).part_bytes + align256(M * r * 2);
}

int64_t mx_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t r) {
  const SkinnyPlan p = plan_skinny(M, K, N, r);
  return p.dz_part + align256(M * r * 2) + p.da_part + p.db_part + align256(K * N * 2) + plan_split16(M, K, N).part_bytes;
}

hipError_t launch_mx_fwd(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, MxView W, const uint16_t* A,
                         const uint16_t* B, float c, uint16_t* Y, uint16_t* Z, void* ws, hipStream_t stream, int dtype) {
  const SkinnyPlan p = plan_skinny(M, K, N, r);
  char* at = static_cast<char*>(ws);
  char* zpart = at + p.at_bytes;
  uint16_t* cbt = reinterpret_cast<uint16_t*>(zpart + p.z_part);
  MxView x{reinterpret_cast<uint8_t*>(cbt) + align256(N * r * 2), nullptr, M, K};
  x.scales = x.codes + align256(mx_code_bytes(M, K));
  uint8_t* part = x.scales + align256(mx_scale_bytes(M, K));
  if (Z == nullptr) Z = reinterpret_cast<uint16_t*>(part + plan_mx(M, N, K).part_bytes);
  const int type = dtype == kDtypeF16 ? NF4_OUT_F16 : NF4_OUT_BF16;
  hipError_t e = launch_mx_quantize(type, false, X, K, x, stream);
  if (e != hipSuccess) return e;
  if ((e = launch_lora_down(M, K, r, X, A, Z, p, at, zpart, stream, N, B, c, cbt, 0, dtype)) != hipSuccess) return e;
  return mx_product(x, W, Z, cbt, r, dtype, type, Y, part, stream);
}

// dX by the dense 16-bit product with the dequantized weight: the gradient's own
// rounding to four bits would be another derivative.
hipError_t launch_mx_bwd(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, const uint16_t* X, Act8View x8,
                         const uint16_t* Z, MxView W, const uint16_t* A, const uint16_t* B, float c, uint16_t* dX,
                         void* dA, void* dB, void* ws, hipStream_t stream, int dtype, bool grad16) {
  const SkinnyPlan p = plan_skinny(M, K, N, r);
  char* dz_part = static_cast<char*>(ws);
  uint16_t* dz16 = reinterpret_cast<uint16_t*>(dz_part + p.dz_part);
  char* da_part = reinterpret_cast<char*>(dz16) + align256(M * r * 2);
  char* db_part = da_part + p.da_part;
  uint16_t* wd = reinterpret_cast<uint16_t*>(db_part + p.db_part);
  hipError_t e = launch_dz(M, N, r, G, B, c, dz16, p, dz_part, stream, dtype);
  if (e != hipSuccess) return e;
  if ((e = launch_colsums(M, K, N, r, X, G, Z, dz16, c, dA, dB, p, da_part, db_part, stream, dtype, grad16, x8)) != hipSuccess)
    return e;
  if (dX == nullptr) return hipGetLastError();
  if ((e = launch_mx_dequantize(dtype == kDtypeF16 ? NF4_OUT_F16 : NF4_OUT_BF16, true, W, wd, N, stream)) != hipSuccess) return e;
  return launch_gated_dx(M, K, N, r, G, wd, dz16, A, dX, stream, dtype, reinterpret_cast<char*>(wd) + align256(K * N * 2));
}

}  // namespace qn
