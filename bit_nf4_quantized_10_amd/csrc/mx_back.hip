// dX = G W + dZ Aᵀ with W (N x K) kept in MXFP4, decoded inside the product, for gfx950:
// calls too small for dequantising W and a dense product by 256 x 256 tiles.
//
// Workgroup: 16 RA rows of G, 128 columns of W and a range of the reduction; its four waves
// take every fourth 32 rows of W.  A lane decodes an 8 x 8 block (a word of codes and a
// scale byte a row), turns it in registers, and has in column t of its block the operand
// of 16 x 16 tile t: no LDS but for the sum of the waves, (0 + 2) + (1 + 3).  The values of
// W are mxfp4_dequantize's, so are their roundings to fp16.  The adapter's product runs as
// more steps of the first range, A's rows read as they lie.
// Bound by the decoding and the waits of two waves a SIMD: 0.6 PFLOP/s at 800 x 4096 x
// 4096, where the dense product of many tiles reaches 1.4.  128 x 8192 x 22016 82 us, each
// block decoded twice, once per 64 rows: vector units 35 %, matrix units 26 %, loads waited
// for 55 % of the waves' time.
#include <hip/hip_ext.h>

#include "common.hpp"
#include "gemv_parts.hpp"
#include "kernels.hpp"
#include "mxfp4.hpp"

namespace qn {

namespace {

constexpr int kBackCols = 128;

struct MxBackArgs {
  const uint16_t *G, *dZ, *A;   // M x N, M x r, K x r
  MxView w;
  int64_t M, N, K, r;
  void* out;                    // M x K in 16 bits, or fp32 planes [splits][M][K]
  int splits, per;              // rows of W a workgroup takes, a multiple of 128
};

template <class T, int RA, bool k16>
__global__ __launch_bounds__(256, 2) void mx_back_kernel(MxBackArgs p) {
  __shared__ f32x4 red[2][RA * 8][64];
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = static_cast<int>(p.M), N = static_cast<int>(p.N), K = static_cast<int>(p.K), r = static_cast<int>(p.r);
  const int strips = (K + kBackCols - 1) / kBackCols, mblocks = (M + 16 * RA - 1) / (16 * RA);
  // row blocks of one piece of W follow each other on one XCD, whose L2 holds it
  const int blk = blockIdx.x, rest = blk >> 3, unit = rest / mblocks * 8 + (blk & 7);
  if (unit >= strips * p.splits) return;
  const int m0 = rest % mblocks * (16 * RA), k0 = unit % strips * kBackCols, split = unit / strips;
  const int nb = static_cast<int>(mx_blocks(K)), chunks = static_cast<int>(mx_chunks(K));
  const Rsrc rc = make_rsrc(p.w.codes, mx_code_bytes(N, K)), rs = make_rsrc(p.w.scales, mx_scale_bytes(N, K));
  const Rsrc rg = make_rsrc(p.G, p.M * p.N * 2), rz = make_rsrc(p.dZ, p.M * p.r * 2), ra = make_rsrc(p.A, p.K * p.r * 2);
  const int k = k0 + 8 * q;
  const uint32_t shift = 8 * ((k0 >> 7) & 3);
  f32x4 acc[RA][8];
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  struct Loads {
    uint32_t c[8];
    uint4 s[2], g[RA];
  };
  const int end = min(N, (split + 1) * p.per);
  auto load = [&](int n0, Loads& L) {   // rows n0 .. n0 + 31; masked past the range's end
    const int n = n0 + 8 * g;
    const bool in = n < end;            // eight rows at once: N and the ranges are multiples of 8
#pragma unroll
    for (int i = 0; i < 8; ++i) L.c[i] = ld_b32(rc, in && k < K ? static_cast<uint32_t>((n + i) * nb) * 16u + k / 2 : kMasked);
    const uint32_t at = static_cast<uint32_t>((n >> 4) * chunks + (k0 >> 9)) * 256u + 4 * (16 * (q >> 2) + 8 * (g & 1));
    L.s[0] = ld_b128(rs, in ? at : kMasked);
    L.s[1] = ld_b128(rs, in ? at + 16 : kMasked);
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      const int m = m0 + 16 * i + q;
      L.g[i] = ld_b128(rg, in && m < M ? (static_cast<uint32_t>(m) * N + n) * 2u : kMasked);
    }
  };
  auto mul = [&](const uint4 (&w)[8], const uint4 (&a)[RA]) {
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < RA; ++i)
        acc[i][t] = T::mfma16(__builtin_bit_cast(typename T::v8, a[i]), __builtin_bit_cast(typename T::v8, w[t]), acc[i][t]);
  };
  auto step = [&](int n0, const Loads& L, Loads& next) {
    load(n0 + 128, next);
    uint4 rows[8], cols[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rows[i] = mx_values8<T>(L.c[i], mx_scale((word_of(L.s[i >> 2], i & 3) >> shift) & 255u));
    transpose8x8_bf16(rows, cols);
    mul(cols, L.g);
  };
  Loads a, b;
  const int beg = split * p.per + 32 * wave;
  load(beg, a);
  for (int n0 = beg; n0 < end; n0 += 256) {
    step(n0, a, b);
    if (n0 + 128 < end) step(n0 + 128, b, a);
  }
  if (split == 0) {
    for (int j0 = 32 * wave; j0 < r; j0 += 128) {
      const int j = j0 + 8 * g;
      uint4 w[8], z[RA];
#pragma unroll
      for (int t = 0; t < 8; ++t) w[t] = ld_b128(ra, j < r && k < K ? (static_cast<uint32_t>(k + t) * r + j) * 2u : kMasked);
#pragma unroll
      for (int i = 0; i < RA; ++i) {
        const int m = m0 + 16 * i + q;
        z[i] = ld_b128(rz, j < r && m < M ? (static_cast<uint32_t>(m) * r + j) * 2u : kMasked);
      }
      mul(w, z);
    }
  }
  // lane: rows 4g + e of tile i, columns 8q .. +7.  The waves' sums, then half of the tiles
  // each to waves 0 and 1.
  if (wave >= 2) {
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
      for (int t = 0; t < 8; ++t) red[wave - 2][8 * i + t][lane] = acc[i][t];
  }
  __syncthreads();
  if (wave < 2) {
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
      for (int t = 0; t < 8; ++t) acc[i][t] += red[wave][8 * i + t][lane];
  }
  __syncthreads();
  if (wave < 2) {
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
      for (int t = 0; t < 8; ++t) red[wave][8 * i + t][lane] = acc[i][t];
  }
  __syncthreads();
  for (int x = wave; x < 4 * RA; x += 4) {   // row 4g + e of tile i
    const int i = x >> 2, e = x & 3, m = m0 + 16 * i + 4 * g + e;
    if (m >= M || k >= K) continue;
    float v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = red[0][8 * i + t][lane][e] + red[1][8 * i + t][lane][e];
    if constexpr (k16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<int64_t>(m) * K + k) =
          make_uint4(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]), T::pack2(v[6], v[7]));
    } else {
      float* o = static_cast<float*>(p.out) + (static_cast<int64_t>(split) * M + m) * K + k;
      *reinterpret_cast<f32x4*>(o) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(o + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
}

template <class T, int RA>
void launch_back_t(const MxBackArgs& p, bool out16, hipStream_t stream, const Timer& tm) {
  const int64_t units = cdiv(p.K, kBackCols) * p.splits, mblocks = cdiv(p.M, 16 * RA);
  const dim3 grid(static_cast<unsigned>(round_up(units, 8) * mblocks));
  hipExtLaunchKernelGGL((out16 ? mx_back_kernel<T, RA, true> : mx_back_kernel<T, RA, false>), grid, dim3(256), 0, stream, tm.start(),
                        tm.end(), 0, p);
}

}  // namespace

// Up to 256 rows, where W's dequantised copy costs most, or 2^33 products.  Whole backward
// this way and by the dense product, us: 1 row, 4096 x 4096 22 and 44; 128 rows, 8192 x
// 22016 115 and 237, 256 180 and 263, 400 298 and 303; 777 x 2056 x 1336 44 and 56; 2048^3
// 57 and 69; 1024 x 4096 x 4096 79 and 84; 333 x 22016 x 2048 99 and 86; 4096 x 512 x 8192
// 115 and 110.
MxBackPlan plan_mx_back(int64_t M, int64_t K, int64_t N) {
  constexpr int64_t kWgs = 512;   // workgroups wanted: two a CU
  MxBackPlan p{};
  if (M > 256 && static_cast<double>(M) * K * N > 8589934592.0) return p;
  const int64_t units = cdiv(K, kBackCols) * cdiv(M, M <= 16 ? 16 : 64), most = cdiv(N, 256);
  int64_t s = kWgs / units;
  s = s < 1 ? 1 : (s > most ? most : s);
  while (s > 1 && s * M * K * 4 > (int64_t(1) << 28)) --s;
  p.per = round_up(cdiv(N, s), 128);
  p.splits = cdiv(N, p.per);
  p.part = p.splits > 1 ? round_up(p.splits * M * K * 4, 256) : 0;
  return p;
}

hipError_t launch_mx_back(const MxBackPlan& pl, int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, const uint16_t* dZ,
                          MxView W, const uint16_t* A, uint16_t* dX, float* part, hipStream_t stream, int dtype) {
  const bool parts = pl.splits > 1;
  const MxBackArgs p{G, dZ, A, W, M, N, K, r, parts ? static_cast<void*>(part) : dX, static_cast<int>(pl.splits), static_cast<int>(pl.per)};
  {
    const Timer tm(QK_BWD_DX, stream, true);
    if (dtype == kDtypeF16) M <= 16 ? launch_back_t<F16, 1>(p, !parts, stream, tm) : launch_back_t<F16, 4>(p, !parts, stream, tm);
    else M <= 16 ? launch_back_t<Bf16, 1>(p, !parts, stream, tm) : launch_back_t<Bf16, 4>(p, !parts, stream, tm);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !parts) return e;
  return launch_split_sum(part, pl.splits, M * K, dX, stream, dtype);
}

}  // namespace qn
