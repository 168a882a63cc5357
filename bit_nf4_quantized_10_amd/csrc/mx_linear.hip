// Products of MXFP4 matrices for gfx950 and the layer on such a weight:
//   C = P Qᵀ (both held in MXFP4),
//   Y = Q(X) Wᵀ + c Z B, Z = X A, and its backward.
// C and Y run on the scaled matrix instructions, whose operand is a lane's block of 32
// elements with its scale (mxfp4.hpp): nothing is decoded.  Many rows run by 256 x 256 tiles
// (mx_core.hpp), few by mx_gemv.hip's kernels.  dX's product is one of 16-bit values, with W
// decoded (below).
//
// Z is rounded to 16 bits once, to what the forward returns and the backward takes: Y's
// adapter term and dB hold the same Z, as in the layer on an NF4 weight.  Against 64 bits
// dB of a bf16 step is off by 0.0024 of its norm, where its own rounding alone is 0.0017; Y's
// 0.0017 does not show it.
#include <hip/hip_ext.h>

#include "common.hpp"
#include "kernels.hpp"
#include "mx_core.hpp"
#include "mxfp4.hpp"

namespace qn {

namespace {

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

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

// Products run by mx_gemv.hip's kernels up to 64 rows or 2^21 outputs, and by tiles above.
// The layer, in a graph: 512 rows at 4096 x 4096 35 us and by tiles 42; 256 rows at
// 4096 x 11008 47 and 42; 777 rows at 2056 x 1336 23 and 33; 1024 at 4096 x 4096 47 and 42.
// Up to 2^17 rows, which the launch that adds their planes and Z's partials takes in one
// grid and with 31-bit offsets.
bool few_rows(int64_t M, int64_t N) { return M <= 64 || (M * N <= (int64_t(1) << 21) && M <= (int64_t(1) << 17)); }

// Splits of a product by tiles (by chunks of the reduction) and their planes' bytes: the
// split of least estimated time, as plan_split16's: rounds of 256 tiles, the planes
// through memory twice and one more launch.  A stage's time is that of few tiles (1.1 us; 1.7
// with all CUs at work, and with that and 9 us a tile the same splits come out at the sizes
// here).  In graphs, split and whole: 2048 x 2048 x 16384 55 and 78 us, 1536 x 1536 x 8192 32
// and 40, 2048 x 2048 x 8192 40 and 41.
struct MxPlan {
  int64_t splits, chunks_per, part_bytes;
};
MxPlan plan_mx(int64_t M, int64_t N, int64_t K) {
  constexpr double kStageUs = 1.2, kTileUs = 5.0, kBytesPerUs = 5e6, kLaunchUs = 4.0;
  const int64_t chunks = mx_chunks(K), tiles = cdiv(M, 256) * cdiv(N, 256), plane = M * N * 4;
  MxPlan pl{1, chunks, 0};
  double least = 2 * kStageUs * chunks + kTileUs;
  if (tiles >= 256) return pl;
  for (int64_t s = 2; s <= chunks && s <= 64 && s * tiles <= 1024; ++s) {
    const int64_t per = cdiv(chunks, s), splits = cdiv(chunks, per);
    if (splits * plane > (int64_t(1) << 28)) break;
    const double us = cdiv(tiles * splits, 256) * (2 * kStageUs * per + kTileUs) + static_cast<double>(splits * plane) * (2.0 / kBytesPerUs) +
                      kLaunchUs + 0.1 * splits;
    if (us >= least) continue;
    least = us;
    pl = MxPlan{splits, per, align256(splits * plane)};
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

hipError_t mx_sum(const float* part, int64_t splits, int64_t count, int out_type, void* out, hipStream_t stream) {
  if (out_type != NF4_OUT_F32)
    return launch_split_sum(part, splits, count, static_cast<uint16_t*>(out), stream, out_type == NF4_OUT_F16 ? kDtypeF16 : kDtypeBf16);
  const int64_t blocks = cdiv(count, 1024);
  Timer tm(QK_REDUCE, stream);
  hipLaunchKernelGGL(mx_sum32_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, part, splits,
                     count, static_cast<float*>(out));
  tm.stop();
  return hipGetLastError();
}

// By tiles.  out_type: NF4_OUT_*; the adapter's operands are of the 16-bit type dtype.
hipError_t mx_tiles(MxView act, MxView w, const uint16_t* ext_a, const uint16_t* ext_b, int64_t r, float c, int dtype, int out_type,
                    void* out, void* ws, hipStream_t stream) {
  const int64_t M = act.rows, N = w.rows;
  const MxPlan pl = plan_mx(M, N, act.cols);
  const bool parts = pl.splits > 1;
  const MxProductArgs p{act, w, ext_a, ext_b, r, c, parts ? ws : out, pl.chunks_per};
  hipError_t e;
  {
    const Timer tm(QK_MX_GEMM, stream, true);
    const bool k32 = parts || out_type == NF4_OUT_F32;
    if (dtype == kDtypeF16) e = k32 ? launch_mx_tiles_t<F16, true>(p, pl.splits, stream, tm) : launch_mx_tiles_t<F16, false>(p, pl.splits, stream, tm);
    else e = k32 ? launch_mx_tiles_t<Bf16, true>(p, pl.splits, stream, tm) : launch_mx_tiles_t<Bf16, false>(p, pl.splits, stream, tm);
  }
  if (e != hipSuccess || !parts) return e;
  return mx_sum(static_cast<const float*>(ws), pl.splits, M * N, out_type, out, stream);
}

}  // namespace

int64_t mx_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return few_rows(M, N) ? plan_mx_rows(M, K, N, 0).part : plan_mx(M, N, K).part_bytes;
}

hipError_t launch_mx_matmul(MxView p, MxView q, int out_type, void* out, void* ws, hipStream_t stream) {
  const int dtype = out_type == NF4_OUT_F16 ? kDtypeF16 : kDtypeBf16;
  if (!few_rows(p.rows, q.rows)) return mx_tiles(p, q, nullptr, nullptr, 0, 0.0f, dtype, out_type, out, ws, stream);
  const MxRowsPlan pl = plan_mx_rows(p.rows, p.cols, q.rows, 0);
  const bool parts = pl.splits > 1;
  hipError_t e = launch_mx_rows(pl, nullptr, &p, q, p.rows, parts ? ws : out, !parts && out_type != NF4_OUT_F32, stream, dtype);
  if (e != hipSuccess || !parts) return e;
  return mx_sum(static_cast<const float*>(ws), pl.splits, p.rows * q.rows, out_type, out, stream);
}

// Workspace of the forward, few rows: the planes, Z's partials, above 16 rows X's codes
// and scales; else: Aᵀ, Z's partials, Bᵀ, X's codes and scales, the tiles' planes.
// Then Z for calls that do not pass it.
static int64_t mx_kept_bytes(int64_t M, int64_t K) { return align256(mx_code_bytes(M, K)) + align256(mx_scale_bytes(M, K)); }
int64_t mx_fwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t r) {
  if (few_rows(M, N)) {
    const MxRowsPlan p = plan_mx_rows(M, K, N, r);
    return p.part + p.zpart + (p.kind != kMxDecode ? mx_kept_bytes(M, K) : 0) + align256(M * r * 2);
  }
  const SkinnyPlan p = plan_skinny(M, K, N, r);
  return p.at_bytes + p.z_part + align256(N * r * 2) + mx_kept_bytes(M, K) + plan_mx(M, N, K).part_bytes + align256(M * r * 2);
}

int64_t mx_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t r) {
  const SkinnyPlan p = plan_skinny(M, K, N, r);
  const MxBackPlan back = plan_mx_back(M, K, N);
  return p.dz_part + 2 * align256(M * r * 2) + p.da_part + p.db_part +
         (back.splits > 0 ? back.part : align256(K * N * 2) + plan_split16(M, K, N).part_bytes);
}

hipError_t launch_mx_fwd(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, MxView W, const uint16_t* A,
                         const uint16_t* B, float c, uint16_t* Y, uint16_t* Z, void* ws, hipStream_t stream, int dtype) {
  const int type = dtype == kDtypeF16 ? NF4_OUT_F16 : NF4_OUT_BF16;
  char* at = static_cast<char*>(ws);
  if (Z == nullptr) Z = reinterpret_cast<uint16_t*>(at + mx_fwd_workspace_bytes(M, K, N, r) - align256(M * r * 2));
  MxView x{nullptr, nullptr, M, K};
  hipError_t e;
  if (few_rows(M, N)) {
    const MxRowsPlan pl = plan_mx_rows(M, K, N, r);
    float* part = reinterpret_cast<float*>(at);
    float* zpart = reinterpret_cast<float*>(at + pl.part);
    const bool decode = pl.kind == kMxDecode;
    if (!decode) {
      x.codes = reinterpret_cast<uint8_t*>(at + pl.part + pl.zpart);
      x.scales = x.codes + align256(mx_code_bytes(M, K));
      if ((e = launch_mx_front(x, X, stream, dtype, &pl, A, r, zpart, nullptr)) != hipSuccess) return e;
    }
    if ((e = launch_mx_rows(pl, X, decode ? nullptr : &x, W, M, part, false, stream, dtype, A, r, zpart)) != hipSuccess) return e;
    return launch_mx_rows_finish(pl, part, zpart, M, N, r, B, c, Y, Z, stream, dtype);
  }
  const SkinnyPlan p = plan_skinny(M, K, N, r);
  char* zpart = at + p.at_bytes;
  uint16_t* bt = reinterpret_cast<uint16_t*>(zpart + p.z_part);
  x.codes = reinterpret_cast<uint8_t*>(bt) + align256(N * r * 2);
  x.scales = x.codes + align256(mx_code_bytes(M, K));
  // Aᵀ and Bᵀ ride along in the launch that quantises X
  TJob tj[2];
  lora_transposes(K, r, A, reinterpret_cast<uint16_t*>(at), N, B, 1.0f, bt, 0, dtype, tj);
  if ((e = launch_mx_front(x, X, stream, dtype, nullptr, nullptr, 0, nullptr, tj)) != hipSuccess) return e;
  if ((e = launch_lora_down(M, K, r, X, A, Z, p, at, zpart, stream, N, B, 1.0f, bt, 0, dtype, true)) != hipSuccess) return e;
  return mx_tiles(x, W, Z, bt, r, c, dtype, type, Y, x.scales + align256(mx_scale_bytes(M, K)), stream);
}

// dX in 16 bits, by the dense product with the dequantized weight or, smaller calls, by
// one that decodes it (mx_back.hip): the gradient's own rounding to four bits would be
// another derivative.  dA takes dZ in two 16-bit parts:
// where few channels of X are far above the others, few rows of dZ make most of dA, and
// dZ's rounding alone would be up to three times dA's own.  In dX, dZ's part is small.
hipError_t launch_mx_bwd(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, const uint16_t* X, Act8View x8,
                         const uint16_t* Z, MxView W, const uint16_t* A, const uint16_t* B, float c, uint16_t* dX,
                         void* dA, void* dB, void* ws, hipStream_t stream, int dtype, bool grad16) {
  const SkinnyPlan p = plan_skinny(M, K, N, r);
  char* dz_part = static_cast<char*>(ws);
  uint16_t* dz16 = reinterpret_cast<uint16_t*>(dz_part + p.dz_part);
  uint16_t* dz_lo = dz16 + align256(M * r * 2) / 2;
  char* da_part = reinterpret_cast<char*>(dz_lo) + align256(M * r * 2);
  char* db_part = da_part + p.da_part;
  uint16_t* wd = reinterpret_cast<uint16_t*>(db_part + p.db_part);
  hipError_t e = launch_dz(M, N, r, G, B, c, dz16, p, dz_part, stream, dtype, nullptr, dz_lo);
  if (e != hipSuccess) return e;
  if ((e = launch_colsums(M, K, N, r, X, G, Z, dz16, c, dA, dB, p, da_part, db_part, stream, dtype, grad16, x8,
                          dz_lo)) != hipSuccess)
    return e;
  if (dX == nullptr) return hipGetLastError();
  const MxBackPlan back = plan_mx_back(M, K, N);
  if (back.splits > 0) return launch_mx_back(back, M, K, N, r, G, dz16, W, A, dX, reinterpret_cast<float*>(wd), stream, dtype);
  if ((e = launch_mx_dequantize(dtype == kDtypeF16 ? NF4_OUT_F16 : NF4_OUT_BF16, true, W, wd, N, stream)) != hipSuccess) return e;
  return launch_gated_dx(M, K, N, r, G, wd, dz16, A, dX, stream, dtype, reinterpret_cast<char*>(wd) + align256(K * N * 2));
}

}  // namespace qn
