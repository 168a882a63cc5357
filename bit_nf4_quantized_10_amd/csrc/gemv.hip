// Small-M forward (M <= 16; the gated block M <= 256) for gfx950: Y = X Ŵ + c Z B as a dequant-GEMV
// (page "QLoRA：冻结的 4-bit 权重怎样参与一次微调", section "量化基座与可训练支路怎样相加";
// the decode is the one of section "Double Quantization 压缩的是 Scale").
//
// Workgroup (4 waves) = two neighbouring 128-column strips x two row ranges;
// each wave streams one strip over its own contiguous range of 32-row steps,
// so the two waves of a row range read the two halves of every 128-byte line
// at about the same time.  Lane (q, g) owns columns n0 + 8q .. +7 and rows
// 8g .. 8g+7 of each step.  Per step a wave stages its codes in LDS (16-byte
// loads of whole 64-byte row pieces), builds the step's 64 block tables
// (32 rows x 2 blocks, 16 RNE(fl32(C[j] * â)) each; one per lane) and
// decodes by table lookups: one byte-select add and one 16-bit LDS read per
// weight, pairs packed with v_perm; column t of the lane feeds the MFMA of
// tile t with the zero-padded 16-row activation block.  A lookup instruction
// touches eight tables that together fill the 64 LDS banks once.  Three
// steps of loads are in flight per wave (per-wave buffer descriptors, so rows
// past the wave's range read as zeros and meet zero activations).  The two
// row ranges of a strip are added in LDS in a fixed order; the split-K
// partials and the LoRA term are added by gemv_finish_kernel.
//
// The gated block's forward for up to 256 rows is the same walk over two weights
// in one launch, its finish forming H = act(G) * U.  Above 16 rows a decoded
// fragment feeds the MFMAs of two or four 16-row tiles (gemv_rows_kernel): a step's
// decode is then shared, and the matrix cores have room (4 to 13 % busy).
// Measured, whole forward, 4096 x 11008: 1 row 24 us, 16 27, 32
// 32, 64 44, 128 74, 256 131; 8192 x 22016: 69, 83, 101, 142, 230, 391.
// No unit is saturated.  One row of 8192 x 22016 (62 us; the codes and scales, 186
// MB, read once at 3.0 TB/s): the waves issue 39 % of their time, wait for loads 25 %
// and hold a ready instruction 37 %, of it 22 % an LDS one; VALU 42 % busy, LDS 21 %
// and 12 % more in bank conflicts.  16 rows of 4096 x 11008, eight steps a wave: the
// CUs hold waves for 59 % of the launch, start and end being the rest, VALU 27 %.
// 100 rows of it: 72 %, 42 % of the waves' time waiting for loads (344 of 512
// workgroups that fit, each weight decoded once per 64 rows).
#include "common.hpp"
#include "gated.hpp"
#include "gemv_parts.hpp"
#include "kernels.hpp"

namespace qn {

namespace {

constexpr int kGvCols = 128;    // columns per workgroup strip (8 per lane)
// Per wave, for one 32-row step: the 64 block tables (32 rows x 2 blocks, 16
// bf16 each) and the step's codes (32 rows x 64 bytes).  The table of row
// 8g + i, block b sits at byte (4i + g) * 64 + 32b, and code row 8g + i at
// (4i + g) * 64, so the 64 lanes of one lookup (rows 8g + i, g < 4, both
// blocks) or of one code read cover the 64 LDS banks once.
constexpr int kGvTabBytes = 32 * 2 * 32;
constexpr int kGvStageBytes = 32 * 64;
constexpr int kGvWaveLds = kGvTabBytes + kGvStageBytes;
#ifndef QN_GV_DEPTH
#define QN_GV_DEPTH 3
#endif
constexpr int kGvDepth = QN_GV_DEPTH;   // 32-row steps of code loads in flight per wave
__device__ __forceinline__ int gv_pos(int row) { return 4 * (row & 7) + (row >> 3); }   // row 8g + i -> 4i + g

// base + byte b of w, one VALU instruction (SDWA byte select on the second operand)
__device__ __forceinline__ uint32_t add_byte(uint32_t base, uint32_t w, int b) {
  uint32_t r;
  switch (b) {
    case 0: asm("v_add_u32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_0" : "=v"(r) : "v"(base), "v"(w)); break;
    case 1: asm("v_add_u32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_1" : "=v"(r) : "v"(base), "v"(w)); break;
    case 2: asm("v_add_u32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_2" : "=v"(r) : "v"(base), "v"(w)); break;
    default: asm("v_add_u32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_3" : "=v"(r) : "v"(base), "v"(w)); break;
  }
  return r;
}

// 16-bit LDS load from a byte address
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  typedef __attribute__((address_space(3))) const uint16_t* lp;
  return *reinterpret_cast<lp>(static_cast<uintptr_t>(addr));
}

template <int R>
struct GvStep {
  uint4 c[2];   // 16 code bytes of one row per load (row order of the LDS stage)
  uint4 x[R];   // activation fragments X[16 rt + q][k + 8g .. k + 8g + 7]
  int q;        // second-level code of the table this lane builds
  float s2;
};

// Workgroup (4 waves) = one 128-column strip; wave w covers rows
// [(split*4 + w) * rpw, +rpw) in steps of 32.  Lane (q, g): columns
// n0 + 8q .. +7, rows 8g .. 8g+7 of each step.  Per step a wave copies its
// 2 KB of codes (two 16-byte loads per lane, whole 64-byte row pieces) into
// its LDS stage, each lane builds one of the step's 64 block tables, and the
// lane reads its eight 4-byte code words back in MFMA order.  Each weight is
// one byte-select add and one 16-bit table lookup, pairs packed with v_perm;
// column t of the lane feeds the MFMA of tile t.  part[split][m][n] = sum of
// the 4 waves (fixed order).
// kTwo: two weights of N columns each (the gated block's), `pairs` strip pairs
// of the first, then of the second; the partials are M x 2N, side by side.
// R > 1 (kTwo only): a workgroup multiplies each decoded fragment with R tiles
// of 16 rows; blocks of 16 R rows are a third factor of the grid.
template <class T, bool kTwo, int R>
__device__ __forceinline__ void gemv_body(const uint16_t* __restrict__ X, int64_t M, NF4View W_, int64_t K, int64_t N,
                                          int64_t rpw, int64_t pairs, float* __restrict__ part,
                                          const uint16_t* __restrict__ A, int64_t r, float* __restrict__ zpart,
                                          NF4View W2) {
  __shared__ float q2t[256];
  __shared__ __attribute__((aligned(16))) char lds[kGvWaves * kGvWaveLds];
  const int t = threadIdx.x, lane = t & 63, q = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t splits = (K + 2 * rpw - 1) / (2 * rpw);
  const int64_t row_pairs = kTwo ? 2 * pairs : pairs;
  const int64_t row_blocks = R > 1 ? (M + 16 * R - 1) / (16 * R) : 1;
  const int64_t gv = row_pairs * splits * row_blocks;
  if (blockIdx.x >= gv) {
    // the last workgroups: Z partials over the same row ranges, 16 rows each
    const int64_t z = blockIdx.x - gv;
    gemv_zpart<T>(X, M, z / splits * 16, K, rpw / 2, A, r, zpart, z % splits, reinterpret_cast<float*>(lds));
    return;
  }
  q2t[t] = q2_value(t - 128);
  // Workgroup ids are dealt to the 8 XCDs in turn.  Logical workgroup L
  // (pair L % pairs of row range L / pairs) is placed so that each XCD runs a
  // contiguous run of L: neighbouring pairs of one row range share an XCD,
  // whose L2 then fetches the lines of int8 scale codes they share once.
  const int64_t per = gv / 8, rem = gv % 8, xcd = blockIdx.x % 8;
  const int64_t L = xcd * per + min(xcd, rem) + blockIdx.x / 8;
  // (row blocks of one strip and row range are neighbours: they decode the same codes)
  const int64_t rb = R > 1 ? L % row_blocks : 0, Ls = R > 1 ? L / row_blocks : L;
  const int64_t row0 = rb * 16 * R;
  const int64_t split = Ls / row_pairs;
  const bool second = kTwo && Ls % row_pairs >= pairs;
  const NF4View W = second ? W2 : W_;
  const int64_t n0 = (2 * (Ls % row_pairs - (second ? pairs : 0)) + (wave & 1)) * kGvCols;
  const int64_t kw0 = (split * 2 + (wave >> 1)) * rpw;
  const int64_t kend = min(K, kw0 + rpw);   // this wave's rows; nothing past them is fetched
  const int64_t rows = kend > kw0 ? kend - kw0 : 0;
  const int64_t kb0 = kend > kw0 ? kw0 : 0;
  // descriptors over this wave's rows only: rows past kend read zeros
  const Rsrc rc = make_rsrc(W.codes + kb0 * N / 2, rows * N / 2);
  // a state without a second level stores one fp32 scale per block: â = that
  const bool single = W.absmax != nullptr;
  const int64_t P = K * N;
  const Rsrc rq = single ? make_rsrc(nullptr, 0) : make_rsrc(W.qabsmax + kb0 * N / 64, rows * N / 64);
  const Rsrc rs = single ? make_rsrc(W.absmax, ((P + 63) / 64) * 4) : make_rsrc(W.absmax2, ((P + 16383) / 16384) * 4);
  const int s_shift = single ? 6 : 14;
  const Rsrc rx = make_rsrc(X, M * K * 2);
  const float off = single ? 0.0f : W.offset[0];
  char* tabs = lds + wave * kGvWaveLds;
  char* stage = tabs + kGvTabBytes;

  // code load j, lane l: stage position p = 16j + l/4 (row 8(p & 3) + p/4),
  // bytes 16(l & 3) .. +15 of that row's 64-byte piece
  uint32_t voff_c[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int p = 16 * j + (lane >> 2), row = 8 * (p & 3) + (p >> 2);
    const int64_t cb = n0 + 32 * (lane & 3);
    voff_c[j] = cb < N ? static_cast<uint32_t>((row * N + cb) >> 1) : kMasked;
  }
  // the table this lane builds: row trow, block tblk of the step
  const int trow = lane >> 1, tblk = lane & 1;
  const int64_t tcol = n0 + 64 * tblk;
  const uint32_t voff_q = tcol < N ? static_cast<uint32_t>((trow * N + tcol) >> 6) : kMasked;
  char* my_tab = tabs + gv_pos(trow) * 64 + 32 * tblk;
  uint32_t voff_x[R];
#pragma unroll
  for (int rt = 0; rt < R; ++rt) {
    const int64_t m = row0 + 16 * rt + q;
    voff_x[rt] = m < M ? static_cast<uint32_t>((m * K + kw0 + 8 * g) * 2) : kMasked;
  }

  auto load = [&](GvStep<R>& S, int64_t kk) {
    // offsets past this wave's rows (or masked) are out of the descriptor: zeros
    const uint32_t sw = static_cast<uint32_t>((kk * N) >> 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) S.c[j] = ld_b128(rc, voff_c[j] + sw);
    // zero activations past this wave's rows (their codes read as 0, a finite weight)
#pragma unroll
    for (int rt = 0; rt < R; ++rt)
      S.x[rt] = ld_b128(rx, (kw0 + kk + 8 * g < kend) ? voff_x[rt] + static_cast<uint32_t>(kk * 2) : kMasked);
    const int64_t kt = kw0 + kk + trow;
    const bool ok = kt < kend && tcol < N;
    S.q = ld_i8(rq, ok ? voff_q + static_cast<uint32_t>((kk * N) >> 6) : kMasked);
    S.s2 = ld_f32(rs, ok ? static_cast<uint32_t>(((kt * N + tcol) >> s_shift) * 4) : kMasked);
  };

  f32x4 acc[R][8];
#pragma unroll
  for (int rt = 0; rt < R; ++rt)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[rt][i] = f32x4{0, 0, 0, 0};
  __syncthreads();  // q2t
  // kDepth steps of loads in flight per wave: set u holds step D j + u and
  // is refilled with step D (j+1) + u as soon as it has been staged.  Each
  // wave's stage and tables are its own, so no workgroup barrier is needed
  // (LDS operations of one wave complete in order).
  constexpr int kDepth = R > 2 ? 2 : kGvDepth;   // four activation fragments a step leave registers for two
  GvStep<R> S[kDepth];
#pragma unroll
  for (int u = 0; u < kDepth; ++u) load(S[u], 32 * u);
  // lookups of row 8g + i go to tbase + 256 i + 2 code
  const uint32_t tbase = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(tabs + g * 64 + 32 * (q >> 3)));
  for (int64_t kk = 0; kk < rpw; kk += 32 * kDepth) {
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int64_t ks = kk + 32 * u;
      if (ks >= rpw) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) *reinterpret_cast<uint4*>(stage + j * 1024 + lane * 16) = S[u].c[j];
      write_block_table<T>(reinterpret_cast<uint16_t*>(my_tab),
                           single ? S[u].s2 : __fadd_rn(__fmul_rn(q2t[S[u].q + 128], S[u].s2), off));
      typename T::v8 xf[R];
#pragma unroll
      for (int rt = 0; rt < R; ++rt) xf[rt] = __builtin_bit_cast(typename T::v8, S[u].x[rt]);
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint32_t*>(stage + (4 * i + g) * 64 + 4 * q);
      load(S[u], ks + 32 * kDepth);   // past the k-range: masked, reads zeros
      // doubled codes: byte b of ev = 2 * code of column 2b, of od = 2 * code
      // of column 2b + 1
      uint32_t ev[8], od[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ev[i] = (w[i] >> 3) & 0x1e1e1e1eu;
        od[i] = (w[i] << 1) & 0x1e1e1e1eu;
      }
#pragma unroll
      for (int tile = 0; tile < 8; ++tile) {
        uint32_t fw[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t a0 = add_byte(tbase, (tile & 1) ? od[2 * p] : ev[2 * p], tile >> 1);
          const uint32_t a1 = add_byte(tbase, (tile & 1) ? od[2 * p + 1] : ev[2 * p + 1], tile >> 1);
          const uint32_t lo = lds_u16(a0 + 2 * p * 256);
          const uint32_t hi = lds_u16(a1 + (2 * p + 1) * 256);
          fw[p] = perm(hi, lo, 0x05040100u);
        }
        const typename T::v8 wf = __builtin_bit_cast(typename T::v8, make_uint4(fw[0], fw[1], fw[2], fw[3]));
#pragma unroll
        for (int rt = 0; rt < R; ++rt) acc[rt][tile] = T::mfma16(xf[rt], wf, acc[rt][tile]);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  // lane holds Y[m = 4g+e][n0 + 8q + tile]; the two row ranges of a strip
  // are added in a fixed order: wave w (w < 2) + wave w + 2
  float* red = reinterpret_cast<float*>(lds);   // 2 waves x 32 floats x 64 lanes = 16 KB
#pragma unroll
  for (int rt = 0; rt < R; ++rt) {
    if (rt > 0) __syncthreads();
    if (wave >= 2) {
#pragma unroll
      for (int tile = 0; tile < 8; ++tile)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[((wave - 2) * 32 + tile * 4 + e) * 64 + lane] = acc[rt][tile][e];
    }
    __syncthreads();
    if (wave < 2) {
      const int64_t ldn = kTwo ? 2 * N : N;
      float* out = part + split * M * ldn + (second ? N : 0);
      const int64_t n = n0 + 8 * q;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = row0 + 16 * rt + 4 * g + e;
        float v[8];
#pragma unroll
        for (int tile = 0; tile < 8; ++tile) v[tile] = acc[rt][tile][e] + red[(wave * 32 + tile * 4 + e) * 64 + lane];
        if (m < M && n < N) {
          *reinterpret_cast<float4*>(out + m * ldn + n) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(out + m * ldn + n + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
  }
}

// Waves per SIMD: three where the registers of one row tile allow it, two above.
template <class T, bool kTwo>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3, 3))) void gemv_kernel(
    const uint16_t* __restrict__ X, int64_t M, NF4View W, int64_t K, int64_t N, int64_t rpw, int64_t pairs,
    float* __restrict__ part, const uint16_t* __restrict__ A, int64_t r, float* __restrict__ zpart, NF4View W2) {
  gemv_body<T, kTwo, 1>(X, M, W, K, N, rpw, pairs, part, A, r, zpart, W2);
}
template <class T, int R>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void gemv_rows_kernel(
    const uint16_t* __restrict__ X, int64_t M, NF4View W, int64_t K, int64_t N, int64_t rpw, int64_t pairs,
    float* __restrict__ part, const uint16_t* __restrict__ A, int64_t r, float* __restrict__ zpart, NF4View W2) {
  gemv_body<T, true, R>(X, M, W, K, N, rpw, pairs, part, A, r, zpart, W2);
}

}  // namespace

#ifndef QN_GV_WAVES
#define QN_GV_WAVES 2752
#endif

void plan_gemv(int64_t M, int64_t K, int64_t N, int64_t r, SkinnyPlan* p_) {
  SkinnyPlan& p = *p_;
  // workgroup = 2 strips x 2 row ranges of rows_per_wave rows, about
  // QN_GV_WAVES waves in total; rows_per_wave is a multiple of 64 so that the Z
  // workgroups' four waves split a row range in 32-row steps
  const int64_t pairs = cdiv(N, 2 * kGvCols);
  const int64_t groups = cdiv(QN_GV_WAVES, pairs * kGvWaves);
  int64_t rpw = round_up(cdiv(K, groups * 2), 64);
  p.gv_rows_per_wave = rpw;
  p.gv_splits = cdiv(K, 2 * rpw);
  p.gv_part = round_up(p.gv_splits * M * N * 4, 256);
  p.gv_zpart = round_up(p.gv_splits * M * r * 4, 256);
}

hipError_t launch_gemv(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, NF4View W, const uint16_t* A,
                       const uint16_t* B, float c, uint16_t* Y, uint16_t* Z, const SkinnyPlan& p, void* part_ws,
                       hipStream_t stream, int dtype) {
  const int64_t pairs = cdiv(N, 2 * kGvCols);
  float* part = static_cast<float*>(part_ws);
  float* zpart = reinterpret_cast<float*>(static_cast<char*>(part_ws) + p.gv_part);
  Timer tm(QK_FWD_GEMV, stream);
  hipLaunchKernelGGL((dtype == kDtypeF16 ? gemv_kernel<F16, false> : gemv_kernel<Bf16, false>), dim3(static_cast<unsigned>((pairs + 1) * p.gv_splits)), dim3(kGvWaves * 64), 0,
                     stream, X, M, W, K, N, p.gv_rows_per_wave, pairs, part, A, r, zpart, W);
  tm.stop();
  Timer te(QK_REDUCE, stream);
  const unsigned phases = static_cast<unsigned>(M < 4 ? M : 4);   // rows 4g + e, e < phases
  hipLaunchKernelGGL((dtype == kDtypeF16 ? gemv_finish_kernel<F16, false, false> : gemv_finish_kernel<Bf16, false, false>), dim3(static_cast<unsigned>(cdiv(N, kFinCols)), phases), dim3(256), 0, stream,
                     static_cast<const float*>(part), static_cast<int>(p.gv_splits), M, N,
                     static_cast<const float*>(zpart), static_cast<int>(p.gv_splits), Z, B, r, c, Y, GatedKeep{});
  te.stop();
  return hipGetLastError();
}

#ifndef QN_GV2_WAVES
#define QN_GV2_WAVES 2752
#endif
// The gated block's two weights share a launch: twice the strips, so half the
// row ranges of one weight's plan; and blocks of 16 R rows.
static int gated_row_tiles(int64_t M) { return M <= 16 ? 1 : (M <= 32 ? 2 : 4); }

// One row tile: about QN_GV2_WAVES waves, which fill the device once (three
// workgroups a CU).  More: the device holds kRowsSlots workgroups at a time (two
// a CU, by registers), and the split is the one with the least estimated time:
// full rounds of workgroups, each kRowsStart us and kRowsStep us per 32-row
// step, then the partials' way through memory.  (Measured at 4096 x 11008, 100
// rows: two row ranges, 358 workgroups in one round, 62 us; three, 537 in two
// rounds, 80 us; at 8192 x 22016, 128 rows: 1.6 us a step.)
constexpr int64_t kRowsSlots = 512;
constexpr double kRowsStart = 4.0, kRowsStep = 1.6, kRowsBytesPerUs = 5e6;
GatedGemvPlan plan_gated_gemv(int64_t M, int64_t K, int64_t F, int64_t r) {
  const int R = gated_row_tiles(M);
  const int64_t units = 2 * cdiv(F, 2 * kGvCols) * cdiv(M, 16 * R);
  int64_t rpw = round_up(cdiv(K, cdiv(QN_GV2_WAVES, units * kGvWaves) * 2), 64);
  if (R > 1) {
    double best = 0.0;
    int64_t last = 0;
    for (int64_t s = 1; s <= 32; ++s) {
      const int64_t rows = round_up(cdiv(K, 2 * s), 64), splits = cdiv(K, 2 * rows);
      if (rows == last) continue;
      if (splits * M * 2 * F * 4 > INT32_MAX) break;   // the finish addresses them with 31-bit offsets; one range always fits
      last = rows;
      const int64_t rounds = cdiv((units + cdiv(M, 16)) * splits, kRowsSlots);
      const double us = static_cast<double>(rounds) * (kRowsStart + kRowsStep * static_cast<double>(rows / 32)) +
                        static_cast<double>(splits * M * 2 * F) * 8.0 / kRowsBytesPerUs;
      if (s == 1 || us < best) {
        best = us;
        rpw = rows;
      }
    }
  }
  const int64_t splits = cdiv(K, 2 * rpw);
  return GatedGemvPlan{rpw, splits, round_up(splits * M * 2 * F * 4, 256), round_up(splits * M * 2 * r * 4, 256)};
}

hipError_t launch_gated_gemv(int64_t M, int64_t K, int64_t F, int64_t r, const uint16_t* X, const NF4View* W,
                             const uint16_t* A, const uint16_t* B, float c, bool gelu, uint16_t* H, uint16_t* Z,
                             const GatedKeep& keep, void* ws, hipStream_t stream, int dtype) {
  const GatedGemvPlan p = plan_gated_gemv(M, K, F, r);
  const int R = gated_row_tiles(M);
  const int64_t pairs = cdiv(F, 2 * kGvCols), tiles = cdiv(M, 16);
  float* part = static_cast<float*>(ws);
  float* zpart = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part);
  auto* k = dtype == kDtypeF16 ? (R == 1 ? gemv_kernel<F16, true> : (R == 2 ? gemv_rows_kernel<F16, 2> : gemv_rows_kernel<F16, 4>))
                               : (R == 1 ? gemv_kernel<Bf16, true> : (R == 2 ? gemv_rows_kernel<Bf16, 2> : gemv_rows_kernel<Bf16, 4>));
  Timer tm(QK_FWD_GEMV, stream);
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>((2 * pairs * cdiv(M, 16 * R) + tiles) * p.splits)),
                     dim3(kGvWaves * 64), 0, stream, X, M, W[0], K, F, p.rows_per_wave, pairs, part, A, 2 * r, zpart,
                     W[1]);
  tm.stop();
  Timer te(QK_REDUCE, stream);
  // rows 4g + e, e < phases, of each tile
  const unsigned phases = static_cast<unsigned>(M < 4 ? M : 4 * tiles);
  auto* fin = dtype == kDtypeF16 ? (gelu ? gemv_finish_kernel<F16, true, true> : gemv_finish_kernel<F16, true, false>)
                                 : (gelu ? gemv_finish_kernel<Bf16, true, true> : gemv_finish_kernel<Bf16, true, false>);
  hipLaunchKernelGGL(fin, dim3(static_cast<unsigned>(cdiv(F, kFinCols / 2)), phases), dim3(256), 0, stream,
                     static_cast<const float*>(part), static_cast<int>(p.splits), M, F,
                     static_cast<const float*>(zpart), static_cast<int>(p.splits), Z, B, r, c, H, keep);
  te.stop();
  return hipGetLastError();
}

}  // namespace qn
