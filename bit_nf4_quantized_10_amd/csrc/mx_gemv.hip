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
#include "mx_offsets.hpp"
#include "mx_quant.hpp"
#include "side_jobs.hpp"

namespace qn {

namespace {

struct MxRowsArgs {
  const uint16_t* X;      // decode kernel: M x K, M <= 16
  MxView act;             // else
  MxView w;
  int64_t M, N, K;
  void* out;              // M x N in 16 bits, or fp32 planes [splits][M][N]
  int splits, chunks_per; // chunks a workgroup takes
  // decode kernel: Z = X A in zsplits more workgroups, z_rpw rows of A a wave
  const uint16_t* A;
  int64_t r;
  float* zpart;
  int zsplits, z_rpw;
};

// In front of a product: X quantised, and the partials of Z = X A in the first workgroups
// (those of 16 rows and one of zsplits ranges of K, or side's transposes).  6 us at 100 x
// 4096, rank 16: a launch and four waits for memory; with 16 ranges instead of 8 the same
// there, and up to 2 us more at one row of 8192 x 22016, whose next launch adds them.
struct MxFrontArgs {
  MxArgs quant;
  const uint16_t* X;
  int64_t M, K, r;
  const uint16_t* A;
  float* zpart;
  int zsplits, z_rpw;
  TJob side[2];
};
template <class T, bool kZ>
__global__ __launch_bounds__(256) void mx_front_kernel(MxFrontArgs p) {
  __shared__ __attribute__((aligned(16))) float lds[kZ ? 4096 : 32 * 33 / 2];
  int64_t blk = blockIdx.x;
  if constexpr (kZ) {
    const int64_t zwgs = p.zsplits * ((p.M + 15) / 16);
    if (blk < zwgs) {
      gemv_zpart<T>(p.X, p.M, blk / p.zsplits * 16, p.K, p.z_rpw, p.A, p.r, p.zpart, blk % p.zsplits, lds);
      return;
    }
    blk -= zwgs;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (blk < p.side[i].nblk) {
        transpose_block(p.side[i], blk, reinterpret_cast<uint16_t(*)[33]>(lds));
        return;
      }
      blk -= p.side[i].nblk;
    }
  }
  mx_quantize_piece<T>(p.quant, blk);
}

template <class T, int RA, int RW, bool k16>
__global__ __launch_bounds__(256) void mx_rows_kernel(MxRowsArgs p) {
  constexpr int kTiles = RA * RW;
  __shared__ f32x4 red[4 * kTiles][64];
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = static_cast<int>(p.M), N = static_cast<int>(p.N), K = static_cast<int>(p.K);
  const int blk = blockIdx.x;
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

// Workgroup: 16 RA activation rows, 64 RW weight rows, 16 RW a wave, and a range of
// chunks.  Weights go from memory into the wave's own fragments (no other wave wants
// them), the chunk's activation codes straight into LDS in the order of the fragments;
// a chunk's loads run while the one before it is multiplied (requested two chunks ahead,
// the weights gained nothing).  At 100 x 4096 x 11008 (15 us) the multiplications and the
// LDS reads alone take 9 with the launch, weights, activations and the fp32 planes 2 to 3
// each.
__device__ __forceinline__ void copy16(Rsrc r, char* to, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(to), 16, voff, soff, 0, 0);
}
constexpr int panel_lds(int ra) { return 2 * 16 * ra * 256; }
template <class T, int RA, int RW, bool k16>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void mx_panel_kernel(MxRowsArgs p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = static_cast<int>(p.M), N = static_cast<int>(p.N), K = static_cast<int>(p.K);
  const int blk = blockIdx.x;
  const int groups = (N + 64 * RW - 1) / (64 * RW), mblocks = (M + 16 * RA - 1) / (16 * RA);
  const int rest = blk >> 3, unit = rest / mblocks * 8 + (blk & 7);   // as mx_rows_kernel
  if (unit >= groups * p.splits) return;
  const int m0 = rest % mblocks * (16 * RA), n0 = unit % groups * (64 * RW) + wave * (16 * RW), split = unit / groups;
  const int nb = static_cast<int>(mx_blocks(K)), chunks = static_cast<int>(mx_chunks(K));
  const int beg = split * p.chunks_per, end = min(beg + p.chunks_per, chunks);
  const Rsrc rw = make_rsrc(p.w.codes, mx_code_bytes(N, K)), rsw = make_rsrc(p.w.scales, mx_scale_bytes(N, K));
  const Rsrc ra = make_rsrc(p.act.codes, mx_code_bytes(M, K)), rsa = make_rsrc(p.act.scales, mx_scale_bytes(M, K));
  uint32_t va[RA];
  // this wave copies step `wave` of the chunk
#pragma unroll
  for (int i = 0; i < RA; ++i)
    va[i] = m0 + 16 * i + q < M ? static_cast<uint32_t>((m0 + 16 * i + q) * nb + 4 * wave + g) * 16u : kMasked;
  struct Loads {
    i32x4 w[RW][4];
    uint32_t sw[RW], sa[RA];
  };
  // Offsets are a lane's own and a scalar, masks in the lane's own (mx_offsets.hpp); tiles
  // past the last one take its scales, for rows that are not stored.
  const int last_w = (N - 1) / 16, last_a = (M - 1) / 16;
  auto load = [&](int c, int buf, Loads& L) {
    const bool in = 16 * c + 4 * wave + g < nb;
#pragma unroll
    for (int i = 0; i < RA; ++i) copy16(ra, smem + buf + (4 * i + wave) * 1024, in ? va[i] : kMasked, 256 * c);
#pragma unroll
    for (int j = 0; j < RW; ++j) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const MxOffset at = mx_code_offset(n0 + 16 * j + q, N, nb, c, s, g);
        L.w[j][s] = __builtin_bit_cast(i32x4, ld128s(rw, at.lane, at.scalar));
      }
      L.sw[j] = ld32s(rsw, 4 * lane, static_cast<uint32_t>(min(n0 / 16 + j, last_w) * chunks + c) * 256u);
    }
#pragma unroll
    for (int i = 0; i < RA; ++i) L.sa[i] = ld32s(rsa, 4 * lane, static_cast<uint32_t>(min(m0 / 16 + i, last_a) * chunks + c) * 256u);
  };
  f32x4 acc[RA][RW];
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RW; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  auto step = [&](int c, int buf, const Loads& L, Loads& next) {
    // this wave's loads of chunk c have landed, and with the barrier everybody's; the
    // other buffer has been read
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (c + 1 < end) load(c + 1, 16 * RA * 256 - buf, next);
    __builtin_amdgcn_sched_barrier(0);
    auto mul = [&](auto tag) {
      constexpr int s = decltype(tag)::value;
      i32x4 fa[RA];
#pragma unroll
      for (int i = 0; i < RA; ++i) fa[i] = *reinterpret_cast<const i32x4*>(smem + buf + (4 * i + s) * 1024 + lane * 16);
#pragma unroll
      for (int i = 0; i < RA; ++i)
#pragma unroll
        for (int j = 0; j < RW; ++j) acc[i][j] = mfma_mx<s>(L.w[j][s], fa[i], acc[i][j], L.sw[j], L.sa[i]);
    };
    mul(std::integral_constant<int, 0>{});
    mul(std::integral_constant<int, 1>{});
    mul(std::integral_constant<int, 2>{});
    mul(std::integral_constant<int, 3>{});
  };
  Loads l0, l1;
  load(beg, 0, l0);
  for (int c = beg; c < end; c += 2) {
    step(c, 0, l0, l1);
    if (c + 1 < end) step(c + 1, 16 * RA * 256, l1, l0);
  }
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      const int m = m0 + 16 * i + q, n = n0 + 16 * j + 4 * g;
      const f32x4& v = acc[i][j];
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
// chunks of their own, 16 rows at 8192 x 22016 took 41 us instead of 27.)  One row of
// 8192 x 22016: 18.8 us, the 96 MB weight at 5.1 TB/s, a copy's rate.
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
  hipExtLaunchKernelGGL((mx_rows_kernel<T, RA, RW, k16>), dim3(static_cast<unsigned>(round_up(units, 8) * mblocks)), dim3(256), 0, stream, tm.start(), tm.end(), 0, p);
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
template <class T, int RA, int RW, bool k16>
hipError_t launch_panel_t(const MxRowsArgs& p, hipStream_t stream, const Timer& tm) {
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&mx_panel_kernel<T, RA, RW, k16>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, panel_lds(RA));
  if (lds_limit != hipSuccess) return lds_limit;
  const dim3 grid(static_cast<unsigned>(round_up(cdiv(p.N, 64 * RW) * p.splits, 8) * cdiv(p.M, 16 * RA)));
  hipExtLaunchKernelGGL((mx_panel_kernel<T, RA, RW, k16>), grid, dim3(256), panel_lds(RA), stream, tm.start(), tm.end(), 0, p);
  return hipGetLastError();
}
template <class T, int RA>
hipError_t launch_panel_r(const MxRowsArgs& p, int rw, bool out16, hipStream_t stream, const Timer& tm) {
  if (rw == 1) return out16 ? launch_panel_t<T, RA, 1, true>(p, stream, tm) : launch_panel_t<T, RA, 1, false>(p, stream, tm);
  return out16 ? launch_panel_t<T, RA, 2, true>(p, stream, tm) : launch_panel_t<T, RA, 2, false>(p, stream, tm);
}
template <class T>
hipError_t launch_panel(const MxRowsArgs& p, int ra, int rw, bool out16, hipStream_t stream, const Timer& tm) {
  return ra == 4 ? launch_panel_r<T, 4>(p, rw, out16, stream, tm) : launch_panel_r<T, 8>(p, rw, out16, stream, tm);
}

constexpr int64_t kWgs = 1024;   // workgroups wanted: four a CU
constexpr int64_t kZSplits = 8;  // of K, in Z's partials

}  // namespace

// Up to this many rows waves take chunks of their own (mx_rows_kernel): 64 x 4096 x 11008
// in 15 us, by panels in 17.
constexpr int64_t kRowsMost = 64;

// r > 0: the layer, whose sums a second launch adds up; else a product alone.
MxRowsPlan plan_mx_rows(int64_t M, int64_t K, int64_t N, int64_t r) {
  MxRowsPlan p{};
  const int64_t chunks = mx_chunks(K);
  // the finish addresses the planes with 31-bit offsets
  auto fits = [&](int64_t s) { return s * M * N * 4 <= INT32_MAX; };
  if (M > kRowsMost) {
    p.kind = kMxPanel;
    // the least estimated time: a start, chunks one after another on a CU (by tiles of 64 or
    // 128 rows and 64 or 128 columns), the planes through memory twice and the launch that adds
    // them; from calls of 64 .. 1024 rows, K 2056 and 4096, N 1336 .. 22016
    constexpr double kStartUs[2][2] = {{6.2, 6.5}, {7.3, 8.2}}, kChunkUs[2][2] = {{1.15, 1.9}, {1.9, 2.1}};
    constexpr double kBytesPerUs = 5e6, kLaunchUs = 4.0;
    double least = 0.0;
    for (int ra = 4; ra <= 8; ra += 4)
      for (int rw = 1; rw <= 2; ++rw)
        for (int64_t s = 1; s <= chunks && s <= 8; ++s) {
          const int64_t per = cdiv(chunks, s);
          if (cdiv(chunks, per) != s || (s > 1 && !fits(s))) continue;
          const int64_t rounds = cdiv(cdiv(N, 64 * rw) * cdiv(M, 16 * ra) * s, 256);
          const double us = kStartUs[ra / 8][rw - 1] + kChunkUs[ra / 8][rw - 1] * static_cast<double>(rounds * per) +
                            (r > 0 || s > 1 ? kLaunchUs + static_cast<double>(s * M * N) * 8.0 / kBytesPerUs : 0.0);
          if (least > 0.0 && us >= least) continue;
          least = us;
          p.ra = ra;
          p.rw = rw;
          p.splits = s;
          p.chunks_per = per;
        }
  } else {
    p.kind = r > 0 && M <= 16 ? kMxDecode : kMxRows;
    p.ra = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
    const int64_t most = p.kind == kMxDecode ? chunks : cdiv(chunks, 4);
    const int64_t wide = p.kind == kMxDecode ? 4 : 1;   // waves side by side
    p.rw = p.ra == 1 ? (cdiv(N, 16 * wide) * most < 2 * kWgs ? 1 : 2) : (p.ra == 2 ? 2 : (cdiv(N, 32) * most < 2 * kWgs ? 2 : 4));
    int64_t s = kWgs / cdiv(N, 16 * wide * p.rw);
    s = s < 1 ? 1 : (s > most ? most : s);
    if (r == 0 && chunks <= 16) s = 1;   // four chunks a wave cost less than the launch that adds planes
    while (s > 1 && !fits(s)) --s;
    p.chunks_per = cdiv(chunks, s);
    p.splits = cdiv(chunks, p.chunks_per);
  }
  if (r > 0) {
    p.z_rpw = round_up(cdiv(K, 4 * kZSplits), 32);
    p.zsplits = cdiv(K, 4 * p.z_rpw);
    p.zpart = round_up(p.zsplits * M * r * 4, 256);
  }
  if (r > 0 || p.splits > 1) p.part = round_up(p.splits * M * N * 4, 256);
  return p;
}

hipError_t launch_mx_front(MxView m, const uint16_t* X, hipStream_t stream, int dtype, const MxRowsPlan* pl, const uint16_t* A, int64_t r,
                           float* zpart, const TJob* side) {
  MxFrontArgs p{};
  p.quant = MxArgs{X, m.cols, m.codes, m.scales, m.rows, m.cols, mx_chunks(m.cols)};
  p.X = X;
  p.M = m.rows;
  p.K = m.cols;
  p.r = r;
  p.A = A;
  p.zpart = zpart;
  int64_t more = 0;
  if (pl != nullptr) {
    p.zsplits = static_cast<int>(pl->zsplits);
    p.z_rpw = static_cast<int>(pl->z_rpw);
    more = pl->zsplits * cdiv(m.rows, 16);
  } else {
    p.side[0] = side[0];
    p.side[1] = side[1];
    more = side[0].nblk + side[1].nblk;
  }
  auto* k = dtype == kDtypeF16 ? (pl != nullptr ? mx_front_kernel<F16, true> : mx_front_kernel<F16, false>)
                               : (pl != nullptr ? mx_front_kernel<Bf16, true> : mx_front_kernel<Bf16, false>);
  Timer tm(QK_MX_QUANT, stream);
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(more + cdiv(m.rows, 16) * p.quant.chunks)), dim3(256), 0, stream, p);
  tm.stop();
  return hipGetLastError();
}

hipError_t launch_mx_rows(const MxRowsPlan& pl, const uint16_t* X, const MxView* act, MxView w, int64_t M, void* out, bool out16,
                          hipStream_t stream, int dtype, const uint16_t* A, int64_t r, float* zpart) {
  const MxRowsArgs p{X, act != nullptr ? *act : MxView{}, w, M, w.rows, w.cols, out, static_cast<int>(pl.splits), static_cast<int>(pl.chunks_per),
                     A, r, zpart, static_cast<int>(pl.zsplits), static_cast<int>(pl.z_rpw)};
  const Timer tm(QK_MX_GEMM, stream, true);
  auto go = [&](auto tag) {
    typedef decltype(tag) T;
    if (pl.kind == kMxPanel) return launch_panel<T>(p, pl.ra, pl.rw, out16, stream, tm);
    if (pl.kind == kMxDecode) launch_decode<T>(p, pl.rw, stream, tm);
    else if (out16) launch_rows_w<T, true>(p, pl.ra, pl.rw, stream, tm);
    else launch_rows_w<T, false>(p, pl.ra, pl.rw, stream, tm);
    return hipGetLastError();
  };
  return dtype == kDtypeF16 ? go(F16{}) : go(Bf16{});
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
