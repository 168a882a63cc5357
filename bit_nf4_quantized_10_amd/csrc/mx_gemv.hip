// Products with an MXFP4 weight for few rows, on gfx950: bound by the one read of the
// weight (0.53 bytes an element).
//
// A workgroup takes 16 RW weight rows and 16 RA activation rows; its four waves take
// every fourth chunk of 512 of the reduction, so that together they read 1 KB of each
// row, and are added in LDS in order.  A wave's operands come straight from memory:
// four steps of v_mfma_scale_f32_16x16x128_f8f6f4 a chunk, each lane one 16-byte block a
// step and tile and one word of scales a chunk (mxfp4.hpp).
// Up to 16 rows of the layer, X is quantised on the way, so the activations cost neither
// a launch nor a pass.
// Few workgroups: the reduction is split over more of them, and the fp32 planes are
// added by the launch that adds the adapter's term (gemv_parts.hpp).
#include <hip/hip_ext.h>

#include "act8.hpp"
#include "common.hpp"
#include "gemv_parts.hpp"
#include "kernels.hpp"
#include "mx_core.hpp"

namespace qn {

namespace {

struct MxRowsArgs {
  const uint16_t* X;      // decode kernel: M x K, M <= 16
  MxView act;             // else
  MxView w;
  int64_t M, N, K;
  void* out;              // M x N in 16 bits, or fp32 planes [splits][M][N]
  int splits, chunks_per; // chunks a workgroup takes
  // Z = X A: zsplits workgroups per 16 rows, z_rpw rows of A a wave (0: none)
  const uint16_t* Xz;
  const uint16_t* A;
  int64_t r;
  float* zpart;
  int zsplits, z_rpw;
};

template <class T, int RA, int RW, bool k16>
__global__ __launch_bounds__(256) void mx_rows_kernel(MxRowsArgs p) {
  constexpr int kTiles = RA * RW;
  __shared__ f32x4 red[4 * kTiles < 16 ? 16 : 4 * kTiles][64];   // 16 KB at least: Z's workgroups use it too
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = static_cast<int>(p.M), N = static_cast<int>(p.N), K = static_cast<int>(p.K);
  const int zwgs = p.zsplits * ((M + 15) / 16), first = (zwgs + 7) & ~7;
  int blk = blockIdx.x;
  if (blk < first) {
    if (blk < zwgs)
      gemv_zpart<T>(p.Xz, p.M, blk / p.zsplits * 16, p.K, p.z_rpw, p.A, p.r, p.zpart, blk % p.zsplits,
                    reinterpret_cast<float*>(red));
    return;
  }
  blk -= first;
  // row blocks of one weight piece follow each other on one XCD (ids are dealt out to
  // the eight in turn), so that its L2 serves all but the first
  const int groups = (N + 16 * RW - 1) / (16 * RW), mblocks = (M + 16 * RA - 1) / (16 * RA);
  const int rest = blk >> 3, unit = rest / mblocks * 8 + (blk & 7);
  if (unit >= groups * p.splits) return;
  const int m0 = rest % mblocks * (16 * RA), n0 = unit % groups * (16 * RW), split = unit / groups;
  const int nb = static_cast<int>(mx_blocks(K)), chunks = static_cast<int>(mx_chunks(K));
  const int beg = split * p.chunks_per, end = min(beg + p.chunks_per, chunks);
  const Rsrc rw = make_rsrc(p.w.codes, mx_code_bytes(N, K)), rsw = make_rsrc(p.w.scales, mx_scale_bytes(N, K));
  const Rsrc ra = make_rsrc(p.act.codes, mx_code_bytes(M, K)), rsa = make_rsrc(p.act.scales, mx_scale_bytes(M, K));
  uint32_t vw[RW], va[RA];
#pragma unroll
  for (int j = 0; j < RW; ++j) vw[j] = n0 + 16 * j + q < N ? static_cast<uint32_t>((n0 + 16 * j + q) * nb + g) * 16u : kMasked;
#pragma unroll
  for (int i = 0; i < RA; ++i) {
    const int m = m0 + 16 * i + q;
    va[i] = m < M ? static_cast<uint32_t>(m * nb + g) * 16u : kMasked;
  }
  f32x4 acc[RA][RW];
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RW; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  for (int c = beg + wave; c < end; c += 4) {
    i32x4 fw[RW][4], fa[RA][4];
    uint32_t sw[RW], sa[RA];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      // tiles past the last one are past the buffer's end: zeros
      sw[j] = ld_b32(rsw, static_cast<uint32_t>((n0 / 16 + j) * chunks + c) * 256u + 4 * lane);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        fw[j][s] = __builtin_bit_cast(i32x4, ld_b128(rw, 16 * c + 4 * s + g < nb ? vw[j] + 256 * c + 64 * s : kMasked));
    }
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      sa[i] = ld_b32(rsa, static_cast<uint32_t>((m0 / 16 + i) * chunks + c) * 256u + 4 * lane);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        fa[i][s] = __builtin_bit_cast(i32x4, ld_b128(ra, 16 * c + 4 * s + g < nb ? va[i] + 256 * c + 64 * s : kMasked));
    }
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        acc[i][j] = mfma_mx<0>(fw[j][0], fa[i][0], acc[i][j], sw[j], sa[i]);
        acc[i][j] = mfma_mx<1>(fw[j][1], fa[i][1], acc[i][j], sw[j], sa[i]);
        acc[i][j] = mfma_mx<2>(fw[j][2], fa[i][2], acc[i][j], sw[j], sa[i]);
        acc[i][j] = mfma_mx<3>(fw[j][3], fa[i][3], acc[i][j], sw[j], sa[i]);
      }
  }
  // lane: act row q of tile i, weight rows 4g .. +3 of tile j
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RW; ++j) red[wave * kTiles + i * RW + j][lane] = acc[i][j];
  __syncthreads();
  for (int x = wave; x < kTiles; x += 4) {
    f32x4 v = red[x][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += red[w * kTiles + x][lane];
    const int m = m0 + 16 * (x / RW) + q, n = n0 + 16 * (x % RW) + 4 * g;
    if (m >= M || n >= N) continue;
    if constexpr (k16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + static_cast<int64_t>(m) * N + n) =
          make_uint2(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]));
    else
      *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + (static_cast<int64_t>(split) * M + m) * N + n) = v;
  }
}

// Up to 16 rows of the layer.  Workgroup: 64 RW weight rows, 16 RW a wave, and a range of
// chunks.  A chunk's 16 x 16 blocks of X are quantised by the 256 threads, a block each
// (maximum, scale and codes need no other lane), and pass through LDS as the operands
// of all four waves; loads of the next chunk are under way meanwhile, across the one
// barrier a chunk.  (With a block's quantisation in every wave that wants it, waves on
// chunks of their own, 16 rows at 8192 x 22016 took 41 us instead of 27.)
template <class T, int RW>
__global__ __launch_bounds__(256) void mx_decode_kernel(MxRowsArgs p) {
  __shared__ __attribute__((aligned(16))) union {
    struct {
      uint4 codes[2][4][64];
      uint32_t scales[2][64];
    } x;
    float red[4096];   // Z's workgroups
  } lds;
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = static_cast<int>(p.M), N = static_cast<int>(p.N), K = static_cast<int>(p.K);
  int blk = blockIdx.x;
  if (blk < p.zsplits) {
    gemv_zpart<T>(p.X, p.M, 0, p.K, p.z_rpw, p.A, p.r, p.zpart, blk, lds.red);
    return;
  }
  blk -= p.zsplits;
  const int groups = (N + 64 * RW - 1) / (64 * RW), split = blk / groups;
  const int n0 = (blk - split * groups) * (64 * RW) + wave * (16 * RW);
  const int nb = static_cast<int>(mx_blocks(K)), chunks = static_cast<int>(mx_chunks(K));
  const int beg = split * p.chunks_per, end = min(beg + p.chunks_per, chunks);
  const Rsrc rw = make_rsrc(p.w.codes, mx_code_bytes(N, K)), rsw = make_rsrc(p.w.scales, mx_scale_bytes(N, K));
  const Rsrc rx = make_rsrc(p.X, p.M * p.K * 2);
  uint32_t vw[RW];
#pragma unroll
  for (int j = 0; j < RW; ++j) vw[j] = n0 + 16 * j + q < N ? static_cast<uint32_t>((n0 + 16 * j + q) * nb + g) * 16u : kMasked;
  // this thread's block: row q, block 4 wave + g of the chunk
  const int bx = 4 * wave + g;
  const uint32_t vx = q < M ? static_cast<uint32_t>(q * K + 32 * bx) * 2u : kMasked;
  struct Loads {
    i32x4 w[RW][4];
    uint32_t sw[RW];
    uint4 x[4];
  };
  auto load = [&](int c, Loads& L) {
#pragma unroll
    for (int k = 0; k < 4; ++k) L.x[k] = ld_b128(rx, 512 * c + 32 * bx + 8 * k < K ? vx + 1024 * c + 16 * k : kMasked);
#pragma unroll
    for (int j = 0; j < RW; ++j) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        L.w[j][s] = __builtin_bit_cast(i32x4, ld_b128(rw, 16 * c + 4 * s + g < nb ? vw[j] + 256 * c + 64 * s : kMasked));
      // tiles past the last one are past the buffer's end: zeros
      L.sw[j] = ld_b32(rsw, static_cast<uint32_t>((n0 / 16 + j) * chunks + c) * 256u + 4 * lane);
    }
  };
  f32x4 acc[RW];
#pragma unroll
  for (int j = 0; j < RW; ++j) acc[j] = f32x4{0, 0, 0, 0};
  auto step = [&](int c, int buf, const Loads& L, Loads& next) {
    const uint32_t m2 = act8_max2(act8_max2(act8_max4(L.x[0]), act8_max4(L.x[1])), act8_max2(act8_max4(L.x[2]), act8_max4(L.x[3])));
    const uint32_t byte = mx_scale_byte(mx_widen_top(T{}, max(m2 & 0xffffu, m2 >> 16)));
    lds.x.codes[buf][wave][lane] = make_uint4(mx_codes8(T{}, L.x[0], byte), mx_codes8(T{}, L.x[1], byte), mx_codes8(T{}, L.x[2], byte),
                                              mx_codes8(T{}, L.x[3], byte));
    reinterpret_cast<uint8_t*>(&lds.x.scales[buf][lane])[wave] = static_cast<uint8_t>(byte);
    if (c + 1 < end) load(c + 1, next);
    // LDS written; loads stay in flight.  (A buffer is written again two barriers on.)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    const uint32_t sa = lds.x.scales[buf][lane];
    i32x4 fa[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) fa[s] = __builtin_bit_cast(i32x4, lds.x.codes[buf][s][lane]);
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      acc[j] = mfma_mx<0>(L.w[j][0], fa[0], acc[j], L.sw[j], sa);
      acc[j] = mfma_mx<1>(L.w[j][1], fa[1], acc[j], L.sw[j], sa);
      acc[j] = mfma_mx<2>(L.w[j][2], fa[2], acc[j], L.sw[j], sa);
      acc[j] = mfma_mx<3>(L.w[j][3], fa[3], acc[j], L.sw[j], sa);
    }
  };
  Loads a, b;
  load(beg, a);
  for (int c = beg; c < end; c += 2) {
    step(c, 0, a, b);
    if (c + 1 < end) step(c + 1, 1, b, a);
  }
  float* out = static_cast<float*>(p.out) + static_cast<int64_t>(split) * M * N;
#pragma unroll
  for (int j = 0; j < RW; ++j) {
    const int n = n0 + 16 * j + 4 * g;
    if (q < M && n < N) *reinterpret_cast<f32x4*>(out + static_cast<int64_t>(q) * N + n) = acc[j];
  }
}

template <class T, int RA, int RW, bool k16>
void launch_rows_t(const MxRowsArgs& p, hipStream_t stream, const Timer& tm) {
  const int64_t units = cdiv(p.N, 16 * RW) * p.splits, mblocks = cdiv(p.M, 16 * RA);
  const int64_t zwgs = round_up(p.zsplits * cdiv(p.M, 16), 8);
  hipExtLaunchKernelGGL((mx_rows_kernel<T, RA, RW, k16>), dim3(static_cast<unsigned>(zwgs + round_up(units, 8) * mblocks)),
                        dim3(256), 0, stream, tm.start(), tm.end(), 0, p);
}
template <class T, bool k16>
void launch_rows_w(const MxRowsArgs& p, int ra, int rw, hipStream_t stream, const Timer& tm) {
  if (ra == 1) {
    if (rw == 1) launch_rows_t<T, 1, 1, k16>(p, stream, tm);
    else launch_rows_t<T, 1, 2, k16>(p, stream, tm);
  } else if (ra == 2) {
    launch_rows_t<T, 2, 2, k16>(p, stream, tm);
  } else {
    if (rw == 2) launch_rows_t<T, 4, 2, k16>(p, stream, tm);
    else launch_rows_t<T, 4, 4, k16>(p, stream, tm);
  }
}
template <class T>
void launch_decode(const MxRowsArgs& p, int rw, hipStream_t stream, const Timer& tm) {
  const dim3 grid(static_cast<unsigned>(p.zsplits + cdiv(p.N, 64 * rw) * p.splits));
  hipExtLaunchKernelGGL((rw == 1 ? mx_decode_kernel<T, 1> : mx_decode_kernel<T, 2>), grid, dim3(256), 0, stream, tm.start(), tm.end(), 0, p);
}

#ifndef QN_MXR_WGS
#define QN_MXR_WGS 512
#endif
#ifndef QN_MXR_ZSPLITS
#define QN_MXR_ZSPLITS 8
#endif

}  // namespace

// r > 0: the layer, whose sums a second launch adds up; else a product alone.
MxRowsPlan plan_mx_rows(int64_t M, int64_t K, int64_t N, int64_t r) {
  MxRowsPlan p{};
  p.ra = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
  p.decode = r > 0 && M <= 16;
  const int64_t chunks = mx_chunks(K), mb = cdiv(M, 16 * p.ra);
  const int64_t most = p.decode ? chunks : cdiv(chunks, 4);
  const int64_t wide = p.decode ? 4 : 1;   // waves side by side
  p.rw = p.ra == 1 ? (cdiv(N, 16 * wide) * most < 2 * QN_MXR_WGS ? 1 : 2) : (p.ra == 2 ? 2 : (cdiv(N, 32) * mb * most < 2 * QN_MXR_WGS ? 2 : 4));
  const int64_t groups = cdiv(N, 16 * wide * p.rw) * mb;
  int64_t s = QN_MXR_WGS / groups;
  s = s < 1 ? 1 : (s > most ? most : s);
  while (s > 1 && s * M * N * 4 > INT32_MAX) --s;   // the finish addresses the planes with 31-bit offsets
  p.chunks_per = cdiv(chunks, s);
  p.splits = cdiv(chunks, p.chunks_per);
  if (r > 0) {
    p.z_rpw = round_up(cdiv(K, 4 * QN_MXR_ZSPLITS), 32);
    p.zsplits = cdiv(K, 4 * p.z_rpw);
    p.zpart = round_up(p.zsplits * M * r * 4, 256);
  }
  if (r > 0 || p.splits > 1) p.part = round_up(p.splits * M * N * 4, 256);
  return p;
}

hipError_t launch_mx_rows(const MxRowsPlan& pl, const uint16_t* X, const MxView* act, MxView w, int64_t M, void* out, bool out16,
                          hipStream_t stream, int dtype, const uint16_t* Xz, const uint16_t* A, int64_t r, float* zpart) {
  const MxRowsArgs p{X, act != nullptr ? *act : MxView{}, w, M, w.rows, w.cols, out, static_cast<int>(pl.splits), static_cast<int>(pl.chunks_per),
                     Xz, A, r, zpart, static_cast<int>(pl.zsplits), static_cast<int>(pl.z_rpw)};
  const Timer tm(QK_MX_GEMM, stream, true);
  auto go = [&](auto tag) {
    typedef decltype(tag) T;
    if (pl.decode) launch_decode<T>(p, pl.rw, stream, tm);
    else if (out16) launch_rows_w<T, true>(p, pl.ra, pl.rw, stream, tm);
    else launch_rows_w<T, false>(p, pl.ra, pl.rw, stream, tm);
  };
  if (dtype == kDtypeF16) go(F16{});
  else go(Bf16{});
  return hipGetLastError();
}

hipError_t launch_mx_rows_finish(const MxRowsPlan& pl, const float* part, const float* zpart, int64_t M, int64_t N, int64_t r,
                                 const uint16_t* B, float c, uint16_t* Y, uint16_t* Z, hipStream_t stream, int dtype) {
  Timer tm(QK_REDUCE, stream);
  const unsigned phases = static_cast<unsigned>(M < 4 ? M : 4 * cdiv(M, 16));   // rows 4g + e, e < phases, of each tile
  hipLaunchKernelGGL((dtype == kDtypeF16 ? gemv_finish_kernel<F16, false, false> : gemv_finish_kernel<Bf16, false, false>),
                     dim3(static_cast<unsigned>(cdiv(N, kFinCols)), phases), dim3(256), 0, stream, part, static_cast<int>(pl.splits), M, N,
                     zpart, static_cast<int>(pl.zsplits), Z, B, r, c, Y, GatedKeep{});
  tm.stop();
  return hipGetLastError();
}

}  // namespace qn
