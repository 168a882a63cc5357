// A 256 x 256-tile core for products of MXFP4 matrices with gfx950's scaled matrix
// instructions: out[m][n] = sum_k act[m][k] w[n][k], fp32 sums, four waves (2 x 2) of
// 128 x 128 each, one wave per SIMD.
//
// It is gemm16.hpp's schedule with 256-element stages: 128 bytes a row as there, so
// the same copies straight from memory to LDS (three slots of activations, two of
// weights, 160 KB) and 16-byte fragments; a stage is two halves of 32 MFMAs over 128
// elements.  v_mfma_scale_f32_32x32x64_f8f6f4 takes the time of a 16-bit one of a
// quarter of its depth, and half a dozen other instructions fit between two of them;
// the 16 x 16 x 128 one with its scales issues twice as often and left no room (1.75
// us a stage).
//
// A lane (i, h) = 32 h + i holds row i of a tile of 32 and in each step one block.  The
// stored order of the scales (mxfp4.hpp) gives it words of blocks g, 4 + g, 8 + g, 12 + g:
// with g = h for the first half of a stage and g = 2 + h for the second, the steps of
// stage p of two take bytes 2p and 2p + 1, and chunks h, 4 + h, 2 + h, 6 + h of the
// rows' eight.  Scales go past LDS, two words a lane and tile for two stages, requested
// two stages ahead.  A tile past the matrix's end takes the last one's scales: its rows
// are not stored.  The adapter's 16-bit product comes first, its few fragments straight
// from memory while the first stages' copies are under way.
//
// Bound by the matrix unit and its power limit in the loop and by bare starts and stores
// around it.  A stage takes 1.7 us with all CUs at work (5.0 PFLOP/s; 4096 x 4096, reductions
// of 2048 to 32768) and 1.1 with a quarter of them, a round of 256 tiles 8 to 10 us besides:
// 4096^3 34 to 37 us (4.0 to 3.7 PFLOP/s), a reduction of 16384 117 to 121 (4.6, the matrix
// unit busy for 76 % of it), 2048 x 8192 x 22016 168; the layer's forward there with an
// adapter of rank 64 206, X's quantisation and Z among it.
#pragma once

#include <type_traits>

#include "gemm16.hpp"
#include "mx_offsets.hpp"
#include "mxfp4.hpp"

namespace qn {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// One 16 x 16 x 128 step, operand bytes `s` of the scales: D[w row 4g + e][act row q].
template <int s>
__device__ __forceinline__ f32x4 mfma_mx(const i32x4& w, const i32x4& a, const f32x4& c, uint32_t sw, uint32_t sa) {
  const i32x8 w8 = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, a8, c, 4, 4, s, static_cast<int>(sw), s, static_cast<int>(sa));
}

// One 32 x 32 x 64 step, in place.  The compiler's own form may put the sum into other
// registers, and with all 256 accumulation registers taken it then moves and spills
// them; the asm ties them.  The s_nop stands for the two wait states that an operand just
// written by a vector instruction needs, which the compiler does not count for asm; what
// reads the sums afterwards waits for the last of them (CoreMx::run).
template <int s>
__device__ __forceinline__ void mfma_mx_in_place(const i32x4& w, const i32x4& a, f32x16& c, uint32_t sw, uint32_t sa) {
#define QN_MX_MFMA(sel) \
  asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 " sel " cbsz:4 blgp:4" \
               : "+a"(c) : "v"(w), "v"(a), "v"(sw), "v"(sa))
  if constexpr (s == 0) QN_MX_MFMA("op_sel_hi:[0,0,0]");
  if constexpr (s == 1) QN_MX_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
  if constexpr (s == 2) QN_MX_MFMA("op_sel_hi:[1,1,0]");
  if constexpr (s == 3) QN_MX_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef QN_MX_MFMA
}

struct MxProductArgs {
  MxView act, w;          // M x K, N x K
  // adapter term, added to the first split: c times ext_a (M x r) times ext_b (N x r)ᵀ
  const uint16_t* ext_a;
  const uint16_t* ext_b;
  int64_t r;
  float c;
  void* out;              // M x N; a split's fp32 planes [splits][M][N]
  int64_t chunks_per;     // 512-element chunks a split takes (all of them: no split)
};

template <class T>
struct CoreMx {
  typedef typename T::v8 v8;
  typedef __attribute__((address_space(3))) char* lds_bytes;
  typedef __attribute__((address_space(3))) const i32x4* lds_frag;
  struct Frags {
    i32x4 a[2][4], w[2][4];      // two steps' tiles
  };
  struct Scales {
    uint32_t a[2][4], w[2][4];   // a stage's halves' tiles
  };

  const MxProductArgs& p;
  char* smem;
  int lane, wave, i32, h, wm, wn;   // lane = 32 h + i32
  // 32-bit and scalar throughout: compares of 64-bit scalars run on the vector units,
  // which drags what they select, descriptors too, into vector registers
  int m0, c0, M, N, nb, chunks;
  Rsrc r_act, r_w, r_sa, r_sw;
  uint32_t av[8], wv[8];       // copies: row wave*64 + 8j + lane/8, chunk_of(j)
  int pA, pW;                  // LDS bytes of fragment 0 at step 0
  uint32_t va[4], vw[4];       // bytes of this lane's scale words of the wave's tiles, chunk 0
  int s_beg, n_full, last;     // first stage, whole stages from it, blocks in front of this share's end
  uint32_t so;

  __device__ CoreMx(const MxProductArgs& args, char* s) : p(args), smem(s) {
    const int t = threadIdx.x;
    lane = t & 63;
    wave = __builtin_amdgcn_readfirstlane(t >> 6);
    i32 = lane & 31;
    h = lane >> 5;
    wm = wave >> 1;
    wn = wave & 1;
    M = static_cast<int>(p.act.rows);
    N = static_cast<int>(p.w.rows);
    nb = static_cast<int>(mx_blocks(p.act.cols));
    chunks = static_cast<int>(mx_chunks(p.act.cols));
    {
      int64_t m, c;
      tile_origin<256>(m, c);
      m0 = static_cast<int>(m);
      c0 = static_cast<int>(c);
    }
    r_act = make_rsrc(p.act.codes, mx_code_bytes(M, p.act.cols));
    r_w = make_rsrc(p.w.codes, mx_code_bytes(N, p.act.cols));
    r_sa = make_rsrc(p.act.scales, mx_scale_bytes(M, p.act.cols));
    r_sw = make_rsrc(p.w.scales, mx_scale_bytes(N, p.act.cols));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = wave * 64 + 8 * j + (lane >> 3);
      const int m = m0 + row, n = c0 + row;
      av[j] = m < M ? static_cast<uint32_t>(m * nb + chunk_of(j)) * 16u : kMasked;
      wv[j] = n < N ? static_cast<uint32_t>(n * nb + chunk_of(j)) * 16u : kMasked;
    }
    const int la = (M - 1) / 16, lw = (N - 1) / 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ia = m0 / 16 + 8 * wm + 2 * i + (i32 >> 4), iw = c0 / 16 + 8 * wn + 2 * i + (i32 >> 4);
      va[i] = static_cast<uint32_t>(min(ia, la) * chunks) * 256u + 4 * (16 * h + (i32 & 15));
      vw[i] = static_cast<uint32_t>(min(iw, lw) * chunks) * 256u + 4 * (16 * h + (i32 & 15));
    }
    pA = (wm * 128 + i32) * 128 + ((h ^ swz(i32)) << 4);
    pW = kG16W + (wn * 128 + i32) * 128 + ((h ^ swz(i32)) << 4);
  }

  // Chunk c of row R lies at c ^ swz(R): 16 lanes' reads, 16 rows of one chunk, fall on
  // all 64 banks once (R & 7 alone took twice the cycles).
  __device__ static int swz(int row) { return (row ^ ((row >> 3) & 3)) & 7; }
  __device__ int chunk_of(int j) const { return (lane & 7) ^ swz(8 * j + (lane >> 3)); }
  __device__ void copy_a(int slot, int j) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r_act, (lds_ptr_t)(smem + slot + (wave * 64 + 8 * j) * 128), 16, av[j], so, 0, 0);
  }
  __device__ void copy_w(int slot, int j) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r_w, (lds_ptr_t)(smem + kG16W + slot + (wave * 64 + 8 * j) * 128), 16, wv[j], so, 0, 0);
  }
  // Points the copies at stage u (counted from s_beg; called for every stage in turn):
  // past the whole stages, blocks past the share's end are masked.  Masks stand in the
  // lanes' own offsets, and the scalar part stays within the rows (mx_offsets.hpp).
  __device__ __forceinline__ void aim(int u) {
    so = mx_stage_offset(s_beg + u, last);
    if (u < n_full) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool past = (s_beg + u) * 8 + chunk_of(j) >= last;
      av[j] = past ? kMasked : av[j];
      wv[j] = past ? kMasked : wv[j];
    }
  }
  // Scale word x of chunk c: of the act (x < 8) or weight tiles, first the words of the
  // stages' first halves.
  __device__ __forceinline__ void load_scale(int c, int x, Scales& S) const {
    const uint32_t at = static_cast<uint32_t>(c) * 256u + ((x >> 2) & 1) * 128u;
    if (x < 8) S.a[(x >> 2) & 1][x & 3] = ld32s(r_sa, va[x & 3], at);
    else S.w[(x >> 2) & 1][x & 3] = ld32s(r_sw, vw[x & 3], at);
  }
  // stage u's chunk, at most the last one
  __device__ int chunk_at(int u) const { return min((s_beg + u) / 2, chunks - 1); }

  // Fragment x (0 .. 15) of a half, in the order of first use: of each of its steps a0,
  // w0 .. w3, a1 .. a3.
  __device__ void read(int sa, int sw, int half, int x, Frags& F) const {
    const lds_bytes base = (lds_bytes)smem;
    const int t = x >> 3, y = x & 7, turn = (t << 6) ^ (half << 5);   // chunk bits 4 and 2
    if (y == 0 || y > 4) {
      const int i = y == 0 ? 0 : y - 4;
      F.a[t][i] = *(lds_frag)(base + (pA ^ turn) + sa + i * 4096);
    } else {
      F.w[t][y - 1] = *(lds_frag)(base + (pW ^ turn) + sw + (y - 1) * 4096);
    }
  }

  // 32 MFMAs from Fc, half kHalf of stage kPart; meanwhile the 16 reads of half `next`
  // into Fn and `side`, called after every MFMA x.
  template <int kPart, int kHalf, class Side>
  __device__ __forceinline__ void half(const Frags& Fc, Frags& Fn, const Scales& S, int sa, int sw, int next, f32x16 (&acc)[4][4],
                                       Side side) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mfma_mx_in_place<2 * kPart>(Fc.w[0][j], Fc.a[0][i], acc[i][j], S.w[kHalf][j], S.a[kHalf][i]);
        __builtin_amdgcn_sched_barrier(0);
        between(sa, sw, next, 4 * i + j, Fn, side);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mfma_mx_in_place<2 * kPart + 1>(Fc.w[1][j], Fc.a[1][i], acc[i][j], S.w[kHalf][j], S.a[kHalf][i]);
        __builtin_amdgcn_sched_barrier(0);
        between(sa, sw, next, 16 + 4 * i + j, Fn, side);
      }
    }
  }
  template <class Side>
  __device__ __forceinline__ void between(int sa, int sw, int next, int x, Frags& Fn, Side side) const {
    if (x < 16) {
      read(sa, sw, next, x, Fn);
      __builtin_amdgcn_sched_barrier(0);
    }
    side(x);
  }
  template <int kInFlight>
  __device__ __forceinline__ static void meet() {
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(kInFlight, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }

  // Stage u from slots sa and sw; the next one's are sa1 and sw1; activations of stage
  // u+2 go to sa2, its weights to sw.  kPart 0, 1: the first and second stage of a chunk
  // with scales S; the first requests the next chunk's into Sn.
  template <int kPart>
  __device__ __forceinline__ void stage(int u, int sa, int sa1, int sa2, int sw, int sw1, Frags& F0, Frags& F1,
                                        const Scales& S, Scales& Sn, f32x16 (&acc)[4][4]) {
    aim(u + 2);
    const int next = chunk_at(u + 2);
    half<kPart, 0>(F0, F1, S, sa, sw, 1, acc, [&](int x) {
      if (x < 16 && (x & 1)) {
        copy_a(sa2, x >> 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (kPart == 0 && x >= 16) {
        load_scale(next, x - 16, Sn);
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    // every wave has read all of stage u (its second half is in registers) and stage
    // u+1 has landed; the copies and scales requested since may be in flight
    meet<kPart == 0 ? 24 : 8>();
    half<kPart, 1>(F1, F0, S, sa1, sw1, 0, acc, [&](int x) {
      if (x < 16 && (x & 1)) {
        copy_w(sw, x >> 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    });
  }

  // 32 of the adapter's rank.
  struct Adapter {
    v8 a[2][4], w[2][4];
  };
  __device__ __forceinline__ void adapter_load(int j0, int r, Adapter& A) const {
    const Rsrc re = make_rsrc(p.ext_a, p.act.rows * p.r * 2), rb = make_rsrc(p.ext_b, p.w.rows * p.r * 2);
    const int stride = static_cast<int>(p.r);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int e = j0 + 16 * t + 8 * h;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + wm * 128 + 32 * i + i32, n = c0 + wn * 128 + 32 * i + i32;
        A.a[t][i] = __builtin_bit_cast(v8, ld_b128(re, m < M && e < r ? static_cast<uint32_t>(m * stride + e) * 2u : kMasked));
        A.w[t][i] = __builtin_bit_cast(v8, ld_b128(rb, n < N && e < r ? static_cast<uint32_t>(n * stride + e) * 2u : kMasked));
      }
    }
  }
  // A sum in vector registers; kFresh: from zero.  s_nop: as mfma_mx_in_place's.
  template <bool kFresh>
  __device__ __forceinline__ static void adapter_mfma(const v8& w, const v8& a, f32x16& x) {
    if constexpr (kFresh) {
      if constexpr (T::kDtype == 1) asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, 0" : "=&v"(x) : "v"(w), "v"(a));
      else asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(x) : "v"(w), "v"(a));
    } else {
      if constexpr (T::kDtype == 1) asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+v"(x) : "v"(w), "v"(a));
      else asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(x) : "v"(w), "v"(a));
    }
  }
  // 64 more of the rank, of which A0 and A1 hold 32 each.
  __device__ __forceinline__ void adapter_add(const Adapter& A0, const Adapter& A1, f32x16 (&acc)[4][4]) const {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const Adapter& A = t < 2 ? A0 : A1;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = T::mfma32(A.w[t & 1][j], A.a[t & 1][i], acc[i][j]);
    }
  }
  // acc = c times the product, whose last 64 (both; else 32) of the rank these are; more: acc
  // holds the others' sums.  c comes in fp32, as in the few rows' path: c B or c Z in 16 bits
  // could pass their range, and a row's result would depend on the rows beside it.  A tile's
  // sum is in vector registers (asm, since the compiler takes accumulation registers, whence
  // all elements are moved to be scaled and back: 2.6 us a round of 256 x 256 tiles more) and
  // scaled while the next two tiles' are computed: behind 32 vector instructions, the first
  // behind four matrix instructions with their waits, where reading it wants 11 wait states.
  // 0.8 us a round more than unscaled: 2048 x 8192 x 22016, rank 64, 203 -> 206 us a call,
  // 4096 x 4096 x 11008, rank 16, 123 -> 126.
  __device__ __forceinline__ void adapter_last(const Adapter& A0, const Adapter& A1, bool more, bool both, f32x16 (&acc)[4][4]) const {
    f32x16 x[3];
#pragma unroll
    for (int k = 0; k < 18; ++k) {
      if (k < 16) {
        f32x16& y = x[k % 3];
        const int i = k >> 2, j = k & 3;
        if (more) {
          y = acc[i][j];
          adapter_mfma<false>(A0.w[0][j], A0.a[0][i], y);
        } else {
          adapter_mfma<true>(A0.w[0][j], A0.a[0][i], y);
        }
        adapter_mfma<false>(A0.w[1][j], A0.a[1][i], y);
        if (both) {
          adapter_mfma<false>(A1.w[0][j], A1.a[0][i], y);
          adapter_mfma<false>(A1.w[1][j], A1.a[1][i], y);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (k >= 2) {
        f32x16& to = acc[(k - 2) >> 2][(k - 2) & 3];
        to = x[(k - 2) % 3] * p.c;
        asm volatile("" : "+a"(to));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // The whole reduction (blockIdx.z's share): clears and fills acc and releases LDS.
  // acc[i][j][4 x + e]: row 32 i + i32 of the wave's 128, column 32 j + 8 x + 4 h + e.  Stages
  // come in pairs, a chunk of scales each; the second of the last pair may be past the end.
  __device__ __forceinline__ void run(f32x16 (&acc)[4][4]) {
    const int beg = static_cast<int>(blockIdx.z) * static_cast<int>(p.chunks_per);
    const int end = min(beg + static_cast<int>(p.chunks_per), chunks);
    s_beg = 2 * beg;
    last = min(16 * end, nb);
    n_full = last / 8 - s_beg;
    Scales S, Sn;
    const int first = chunk_at(0);
    // the adapter's first 64, requested before the copies: loads land in order
    const int r = blockIdx.z == 0 ? static_cast<int>(p.r) : 0;
    Adapter A0, A1;
    if (r > 0) {
      adapter_load(0, r, A0);
      adapter_load(32, r, A1);
    }
#pragma unroll
    for (int x = 0; x < 16; ++x) load_scale(first, x, S);
    aim(0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      copy_a(0, j);
      copy_w(0, j);
    }
    aim(1);
#pragma unroll
    for (int j = 0; j < 8; ++j) copy_a(kTileBytes, j);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        asm volatile("" : "+a"(acc[i][j]));
      }
    if (r > 0) {
#pragma unroll 1
      for (int j0 = 64; j0 < r; j0 += 64) {
        adapter_add(A0, A1, acc);
        adapter_load(j0, r, A0);
        adapter_load(j0 + 32, r, A1);
        // here, so that a rank of up to 64 waits below for its own loads alone, not for as many
        // as this loop would leave under way
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
      }
      adapter_last(A0, A1, r > 64, r > 32, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
    Frags F0, F1;
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 0));
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int x = 0; x < 16; ++x) read(0, 0, 0, x, F0);
#pragma unroll
    for (int j = 0; j < 8; ++j) copy_w(kTileBytes, j);
    int sa = 0, sa1 = kTileBytes, sa2 = 2 * kTileBytes;
    for (int u = 0; u < 2 * (end - beg); u += 2) {
      // two stages: the weights' slots are back where they were, the activations' moved on twice
      stage<0>(u, sa, sa1, sa2, 0, kTileBytes, F0, F1, S, Sn, acc);
      stage<1>(u + 1, sa1, sa2, sa, kTileBytes, 0, F0, F1, S, Sn, acc);
      S = Sn;
      const int s = sa;
      sa = sa2;
      sa2 = sa1;
      sa1 = s;
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    // the last products' results, and the sums in accumulation registers up to here
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
  }

  // The tile in 16 bits, through LDS so that every store is of whole lines.
  __device__ __forceinline__ void store16(const f32x16 (&acc)[4][4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int R = wm * 128 + 32 * i + i32;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int c = wn * 16 + 4 * j + x;
          const f32x16& v = acc[i][j];
          *reinterpret_cast<uint2*>(smem + R * 512 + ((c ^ i32) << 4) + 8 * h) =
              make_uint2(T::pack2(v[4 * x], v[4 * x + 1]), T::pack2(v[4 * x + 2], v[4 * x + 3]));
        }
    }
    __syncthreads();
    const int c = lane & 31;
    const int col = c0 + 8 * c;
#pragma unroll 4
    for (int u = 0; u < 32; ++u) {
      const int R = wave * 64 + 2 * u + (lane >> 5);
      const uint4 v = *reinterpret_cast<const uint4*>(smem + R * 512 + ((c ^ (R & 31)) << 4));
      if (m0 + R < M && col < N)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v),
                                    reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + static_cast<int64_t>(m0 + R) * N + col));
    }
  }
  // In fp32, into this split's plane.
  __device__ __forceinline__ void store32(const f32x16 (&acc)[4][4]) const {
    const Rsrc ro = make_rsrc(static_cast<float*>(p.out) + (static_cast<int64_t>(blockIdx.z) * M + m0) * N + c0,
                              (static_cast<int64_t>(M - m0) * N - c0) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = wm * 128 + 32 * i + i32;
      const bool row_ok = m0 + row < M;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int col = wn * 128 + 32 * j + 8 * x + 4 * h;
          const f32x16& v = acc[i][j];
          const uint32_t voff = row_ok && c0 + col < N ? static_cast<uint32_t>(row) * (4u * N) + 4u * col : kMasked;
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]}), ro,
                                                 voff, 0, 0);
        }
    }
  }
};

}  // namespace

}  // namespace qn
