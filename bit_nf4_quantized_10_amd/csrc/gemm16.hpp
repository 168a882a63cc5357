// A 256 x 256-tile GEMM core on 16 x 16 x 32 MFMAs, for the kernels of the gated
// block and the output head: out[m][n] = sum_k act[m][k] w[n][k], fp32 sums,
// four waves (2 x 2) of 128 x 128 each, one wave per SIMD.
//
// 64-element stages go through three LDS slots of activations and two of
// weights (256 rows of 128 bytes each, the whole 160 KB); 16-byte chunk c of
// row R lies at c ^ (R & 7), which keeps the fragment reads free of bank
// conflicts.  A stage is two halves of 64 MFMAs over 32 elements.  In each the
// next half's fragments (8 of each operand, a second register set) are read
// and copies for stage u+2 go straight from memory to LDS: activations in the
// first half, weights in the second, after the stage's one barrier.
//
// What makes it fast is how little else a wave issues.  One 16-cycle MFMA
// leaves room for three other instructions, and a gap that holds more stalls
// the matrix pipe.  So fragments lie at one address register plus immediate
// offsets, copies carry no masks (where the product's whole stages end, a rare
// branch rewrites the copies' own offsets), and reads and copies are spread over
// the MFMAs: 75 instructions for 128 of them.
// At 4096 x 4096 x 11008 on random bf16 it takes 237 us (1.56 PFLOP/s, 1.47 at
// 4096^3) against 264 us for the same tile on 32 x 32 x 16 MFMAs; on zeros, where
// the power limit does not bind, 172 against 180.
#pragma once

#include "gemm_core.hpp"

namespace qn {

namespace {

// Where a stage's 256 weight rows come from.
//   kRows:   rows c0 .. c0 + 255 of w (wrows x red);
//   kPaired: w stacks two weights of wrows / 2 rows; a tile takes 128 rows of
//     the first and the same 128 of the second, and each wave 64 of both, so a
//     lane holds the pair of values of an element (tiles j and j + 4);
//   kTurned: w is red x wrows.  Its 64 x 256 block of a stage passes through
//     registers: thread (vg, cg) loads rows 8 vg .. +7, columns 8 cg .. +7, turns
//     them with byte permutes and writes them as chunks.  (Transposing LDS reads
//     instead move half the bytes a cycle and made the loop twice as slow.)
enum { kRows = 0, kPaired = 1, kTurned = 2 };

struct G16Args {
  const uint16_t* act;     // M x red, row stride act_ld
  int64_t act_ld;
  const uint16_t* w;
  int64_t w_ld;            // kRows, kPaired: w's row stride
  int64_t M, wrows, red;
  // Adapter term, as more stages after the product's: kRows: ext_a (M x r) times
  // ext_b (wrows x r)ᵀ.  kPaired: ext_a is M x 4r, [hi | lo] parts of the two
  // weights' Z, and each weight's rows of ext_b meet their own Z in both parts.
  const uint16_t* ext_a;
  int64_t ext_a_ld;
  const uint16_t* ext_b;
  int64_t r;
  // Split reduction (part non-null): workgroup z takes elements [z k_per,
  // (z+1) k_per); only z = 0 adds the adapter term.
  float* part;
  int64_t k_per;
  int64_t first = 0;       // column of the launch's first tile (a multiple of kCols)
};

constexpr int kG16W = 3 * kTileBytes;      // the weight slots follow the activation slots
constexpr int kG16Lds = 5 * kTileBytes;

// Rows 2p and 2p + 1 of column c of the 8 x 8 block of 16-bit values `in` (one
// uint4 a row).
__device__ __forceinline__ uint32_t column2(const uint4 (&in)[8], int c, int p) {
  const uint4 &lo = in[2 * p], &hi = in[2 * p + 1];
  const int w = c >> 1;
  const uint32_t l = w == 0 ? lo.x : (w == 1 ? lo.y : (w == 2 ? lo.z : lo.w));
  const uint32_t h = w == 0 ? hi.x : (w == 1 ? hi.y : (w == 2 ? hi.z : hi.w));
  return __builtin_amdgcn_perm(h, l, (c & 1) ? 0x07060302u : 0x05040100u);
}

template <class T, int kW>
struct Core16 {
  static constexpr int kCols = kW == kPaired ? 128 : 256;   // output columns a tile advances by
  typedef typename T::v8 v8;
  typedef __attribute__((address_space(3))) char* lds_bytes;
  typedef __attribute__((address_space(3))) const v8* lds_frag;
  struct Frags {
    v8 a[8], w[8];
  };

  const G16Args& a;
  char* smem;
  int t, lane, wave, q, g, wm, wn;   // lane = 16 g + q
  int64_t m0, c0;
  Rsrc r_act, r_w, r_ea, r_eb;
  uint32_t av[8], wv[8];       // copies: row wave*64 + 8j + lane/8, chunk (lane & 7) ^ (lane >> 3)
                               // (kTurned: wv[i] is row i of this thread's 8 x 8 block)
  int chunk8;                  // 8 * that chunk
  int pA, pW;                  // LDS bytes of fragment 0 at half 0
  int wdst;                    // kTurned: where the turned block goes
  int64_t s_beg, n_main, n_full, r_ext;
  uint32_t so, so_w;           // scalar byte offsets of the next copies and, kTurned, weight loads

  __device__ Core16(const G16Args& args, char* s) : a(args), smem(s) {
    t = threadIdx.x;
    lane = t & 63;
    wave = __builtin_amdgcn_readfirstlane(t >> 6);
    q = lane & 15;
    g = lane >> 4;
    wm = wave >> 1;
    wn = wave & 1;
    tile_origin<kCols>(m0, c0);
    c0 += a.first;
    r_act = make_rsrc(a.act, ((a.M - 1) * a.act_ld + (a.red + 7) / 8 * 8) * 2);   // whole chunks
    r_w = make_rsrc(a.w, (kW == kTurned ? a.red * a.wrows : a.wrows * a.w_ld) * 2);
    r_ea = make_rsrc(a.ext_a, a.r ? a.M * a.ext_a_ld * 2 : 0);
    r_eb = make_rsrc(a.ext_b, a.wrows * a.r * 2);
    chunk8 = 8 * ((lane & 7) ^ (lane >> 3));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = wave * 64 + 8 * j + (lane >> 3);
      const int64_t m = m0 + row, n = weight_row(row);
      av[j] = m < a.M ? static_cast<uint32_t>((m * a.act_ld + chunk8) * 2) : kMasked;
      if (kW != kTurned) wv[j] = n < a.wrows ? static_cast<uint32_t>((n * a.w_ld + chunk8) * 2) : kMasked;
    }
    pA = (wm * 128 + q) * 128 + ((g ^ (q & 7)) << 4);
    const int wrow = (kW == kPaired ? wn * 64 : wn * 128) + q;
    pW = kG16W + wrow * 128 + ((g ^ wswz(wrow)) << 4);
    if (kW == kTurned) {
      const int vg = t >> 5, cg = t & 31;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        wv[i] = c0 + 8 * cg < a.wrows ? static_cast<uint32_t>(((8 * vg + i) * a.wrows + c0 + 8 * cg) * 2) : kMasked;
      wdst = kG16W + 8 * cg * 128 + (((vg ^ cg) & 7) << 4);   // column c: + 128 c, chunk bits ^ c
    }
  }
  // kTurned writes a column of 8 rows at a time, 8 columns apart: the swizzle
  // takes in row >> 3 so that they fall on different banks.
  __device__ static int wswz(int row) { return kW == kTurned ? (row ^ (row >> 3)) & 7 : row & 7; }
  // Row of w that the tile's weight row `row` (0 .. 255) takes; at or past wrows
  // where there is none.
  __device__ int64_t weight_row(int row) const {
    if (kW != kPaired) return c0 + row;
    const int64_t half = a.wrows >> 1, col = c0 + (row & 127);
    return col < half ? (row < 128 ? col : half + col) : a.wrows;
  }

  // Copies of the stage aim() was last called for to byte `slot` of LDS.
  __device__ void copy_a(int slot, int j) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r_act, (lds_ptr_t)(smem + slot + (wave * 64 + 8 * j) * 128), 16, av[j], so, 0, 0);
  }
  __device__ void copy_w(int slot, int j) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r_w, (lds_ptr_t)(smem + kG16W + slot + (wave * 64 + 8 * j) * 128), 16, wv[j], so, 0, 0);
  }
  // Points the copies at stage u (counted from s_beg; called for every stage in
  // turn).  Past the product's whole stages: the chunks past the reduction's end
  // are masked, then come the adapter's stages, then nothing.  Every mask is in the
  // lane's own offset and no scalar offset passes its operand's end, since a
  // buffer's range check need not count the scalar part.
  __device__ __forceinline__ void aim(int64_t u) {
    so = static_cast<uint32_t>((s_beg + u) * (kBK * 2));
    if (kW == kTurned) so_w = static_cast<uint32_t>(s_beg + u) * static_cast<uint32_t>(a.wrows * (kBK * 2));
    if (u < n_full) return;
    // One assignment per offset, whichever case holds (stores that the compiler
    // merges from two branches would keep the arrays in memory), and descriptors
    // that change in uniform control flow only.
    const bool tail = u < n_main;
    const bool past = (s_beg + u) * kBK + chunk8 >= a.red;
    const int64_t e = (u - n_main) * kBK + chunk8;
    if (!tail) {
      so = 0;
      so_w = 0;
      r_act = r_ea;
      if (kW != kTurned) r_w = r_eb;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = wave * 64 + 8 * j + (lane >> 3);
      const int64_t m = m0 + row;
      const uint32_t ea = m < a.M && e < r_ext ? static_cast<uint32_t>((m * a.ext_a_ld + e) * 2) : kMasked;
      av[j] = tail ? (past ? kMasked : av[j]) : ea;
      if (kW == kTurned) {
        wv[j] = tail && (s_beg + u) * kBK + 8 * (t >> 5) + j < a.red ? wv[j] : kMasked;
        continue;
      }
      const int64_t n = weight_row(row);
      int64_t own = e;   // within this row's own r
      if (kW == kPaired) own = (e >= 2 * a.r ? e - 2 * a.r : e) - (row < 128 ? 0 : a.r);
      const uint32_t eb =
          n < a.wrows && e < r_ext && own >= 0 && own < a.r ? static_cast<uint32_t>((n * a.r + own) * 2) : kMasked;
      wv[j] = tail ? (past ? kMasked : wv[j]) : eb;
    }
  }
  // kTurned: row 8 vg + i of the stage aim() was last called for (zeros past this
  // workgroup's rows)
  __device__ uint4 load_w(int i) const { return ld128s(r_w, wv[i], so_w); }
  // kTurned: writes column c of the registers' block to weight slot `slot`.  As
  // an instruction: for a plain store the compiler first waits for every copy
  // still in flight, since one could write the same LDS bytes (none does).  The
  // writes are waited for before the barrier (lgkmcnt); waits the compiler sets
  // for its own LDS reads count them as well and so only come out longer.
  __device__ void put_w(uint32_t d0, uint32_t d1, uint32_t d2, uint32_t d3, int slot, int c) const {
    const u32x4 d = {d0, d1, d2, d3};
    const uint32_t at = (wdst ^ (c << 4)) + (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem)) + slot + 128 * c);
    asm volatile("ds_write_b128 %0, %1" ::"v"(at), "v"(d) : "memory");
  }
  __device__ void store_w(const uint4 (&R)[8], int slot, int c) const {
    put_w(column2(R, c, 0), column2(R, c, 1), column2(R, c, 2), column2(R, c, 3), slot, c);
  }

  // Addresses of a half's fragments.
  struct Place {
    int a, w[kW == kTurned ? 4 : 1];
  };
  __device__ Place place(int sa, int sw, int half) const {
    Place p;
    p.a = (pA ^ (half << 6)) + sa;
    if (kW == kTurned) {
#pragma unroll
      for (int x = 0; x < 4; ++x) p.w[x] = (pW ^ (((x ^ (half << 1)) & 3) << 5)) + sw;
    } else {
      p.w[0] = (pW ^ (half << 6)) + sw;
    }
    return p;
  }
  // Fragment x in the order of first use: a0, w0 .. w7, a1 .. a7.
  __device__ void read(const Place& p, int x, Frags& F) const {
    const lds_bytes base = (lds_bytes)smem;
    if (x == 0 || x > 8) {
      const int i = x == 0 ? 0 : x - 8;
      F.a[i] = *(lds_frag)(base + p.a + i * 2048);
    } else {
      const int j = x - 1;
      const int at = kW == kPaired ? (j >> 2) * 16384 + (j & 3) * 2048 : j * 2048;
      F.w[j] = *(lds_frag)(base + p.w[kW == kTurned ? j & 3 : 0] + at);
    }
  }

  // 64 MFMAs from Fc; meanwhile the 16 reads at p into Fn and `side`, called
  // after every MFMA (i, j).  The order is pinned with scheduling barriers.
  template <class Side>
  __device__ __forceinline__ void half(const Frags& Fc, Frags& Fn, const Place& p, f32x4 (&acc)[8][8], Side side) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[i][j] = T::mfma16(Fc.w[j], Fc.a[i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
        // kTurned: after its other work
        const int x = kW == kTurned ? (i >= 2 && j < 6 ? 3 * (i - 2) + (j >> 1) : 16) : 4 * i + (j >> 1);
        if ((j & 1) && x < 16) {
          read(p, x, Fn);
          __builtin_amdgcn_sched_barrier(0);
        }
        side(i, j);
      }
    }
  }
  template <int kInFlight>
  __device__ __forceinline__ static void meet() {
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(kInFlight, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }

  // Stage u from slots sa and sw; the next one's are sa1 and sw1; activations of
  // stage u+2 go to sa2, its weights to sw.
  __device__ __forceinline__ void stage(int64_t u, int sa, int sa1, int sa2, int sw, int sw1, Frags& F0, Frags& F1,
                                        f32x4 (&acc)[8][8]) {
    aim(u + 2);
    half(F0, F1, place(sa, sw, 1), acc, [&](int i, int j) {
      if ((j & 3) == 2 && i < 4) {
        copy_a(sa2, 2 * i + (j >> 2));
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    // every wave has read all of stage u (its second half is in registers) and
    // stage u+1 has landed; the 8 copies of stage u+2 may be in flight
    meet<8>();
    half(F1, F0, place(sa1, sw1, 0), acc, [&](int i, int j) {
      if ((j & 3) == 2 && i < 4) {
        copy_w(sw, 2 * i + (j >> 2));
        __builtin_amdgcn_sched_barrier(0);
      }
    });
  }
  // kTurned: the first half writes the weights of stage u+1 from R to sw1 during
  // its first 16 MFMAs, requests those of stage u+2 into R (most of a stage ahead
  // of their use) and copies the activations of stage u+2.
  __device__ __forceinline__ void stage_turned(int64_t u, int sa, int sa1, int sa2, int sw, int sw1, Frags& F0, Frags& F1,
                                               uint4 (&R)[8], f32x4 (&acc)[8][8]) {
    aim(u + 2);
    uint32_t d[4];
    half(F0, F1, place(sa, sw, 1), acc, [&](int i, int j) {
      if (i < 2) {
        const int c = 4 * i + (j >> 1);
        if ((j & 1) == 0) {
#pragma unroll
          for (int p = 0; p < 4; ++p) d[p] = column2(R, c, p);
        } else {
          put_w(d[0], d[1], d[2], d[3], sw1, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      } else if (i < 4 && (j & 1) == 0) {
        R[4 * (i - 2) + (j >> 1)] = load_w(4 * (i - 2) + (j >> 1));
        __builtin_amdgcn_sched_barrier(0);
      } else if (i >= 4 && (j & 3) == 2) {
        copy_a(sa2, 2 * (i - 4) + (j >> 2));
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    // the weights of stage u+1 are written, its activations have landed; the
    // weights and the activations of stage u+2 may be in flight
    meet<16>();
    half(F1, F0, place(sa1, sw1, 0), acc, [](int, int) {});
  }

  // The whole reduction (kSplit: blockIdx.z's share): clears and fills acc and
  // releases LDS.  acc[i][j]: rows 16 i + q of the wave's 128, columns 16 j + 4 g
  // .. +3 (kPaired: 16 (j & 3) + 4 g of the wave's 64, of the second weight for
  // j >= 4).
  template <bool kSplit>
  __device__ __forceinline__ void run(f32x4 (&acc)[8][8]) {
    const int64_t all = (a.red + kBK - 1) / kBK;
    s_beg = 0;
    int64_t end = all;
    if (kSplit) {
      s_beg = static_cast<int64_t>(blockIdx.z) * (a.k_per / kBK);
      end = s_beg + a.k_per / kBK < all ? s_beg + a.k_per / kBK : all;
    }
    n_main = end - s_beg;
    n_full = (a.red / kBK < end ? a.red / kBK : end) - s_beg;
    r_ext = !kSplit || blockIdx.z == 0 ? (kW == kPaired ? 4 * a.r : a.r) : 0;
    const int64_t total = n_main + (r_ext + kBK - 1) / kBK;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    Frags F0, F1;
    int sa = 0, sa1 = kTileBytes, sa2 = 2 * kTileBytes, sw = 0;
    auto turn = [&] {
      const int s = sa;
      sa = sa1;
      sa1 = sa2;
      sa2 = s;
      sw ^= kTileBytes;
    };
    if constexpr (kW == kTurned) {
      uint4 R[8];
      aim(0);
#pragma unroll
      for (int i = 0; i < 8; ++i) R[i] = load_w(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) copy_a(0, j);
#pragma unroll
      for (int c = 0; c < 8; ++c) store_w(R, 0, c);
      aim(1);
#pragma unroll
      for (int i = 0; i < 8; ++i) R[i] = load_w(i);   // in the order of the loop's own loads, whose waits the compiler counts
#pragma unroll
      for (int j = 0; j < 8; ++j) copy_a(kTileBytes, j);
      __builtin_amdgcn_s_waitcnt(waitcnt_imm(16, 0));   // stage 0; the 16 loads since may be in flight
      __builtin_amdgcn_s_barrier();
      const Place p = place(0, 0, 0);
#pragma unroll
      for (int x = 0; x < 16; ++x) read(p, x, F0);
      for (int64_t u = 0; u < n_main; ++u, turn()) stage_turned(u, sa, sa1, sa2, sw, sw ^ kTileBytes, F0, F1, R, acc);
    } else {
      aim(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        copy_a(0, j);
        copy_w(0, j);
      }
      aim(1);
#pragma unroll
      for (int j = 0; j < 8; ++j) copy_a(kTileBytes, j);
      __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 0));
      __builtin_amdgcn_s_barrier();
      const Place p = place(0, 0, 0);
#pragma unroll
      for (int x = 0; x < 16; ++x) read(p, x, F0);
#pragma unroll
      for (int j = 0; j < 8; ++j) copy_w(kTileBytes, j);
      for (int64_t u = 0; u < total; ++u, turn()) stage(u, sa, sa1, sa2, sw, sw ^ kTileBytes, F0, F1, acc);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    // Keeps the sums in accumulation registers up to here: an epilogue that works
    // on many of them at once would otherwise draw some into the vector registers
    // for the whole loop, at the price of moves in it.
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
  }

  // The tile as 16-bit rows of 256 columns through LDS, so that every store is
  // of whole lines: put16 for each (i, j), then flush16 with store8(row of the
  // tile, 16-byte group of 8 columns, values).
  __device__ __forceinline__ void put16(int i, int j, float v0, float v1, float v2, float v3) const {
    const int R = wm * 128 + 16 * i + q;
    const int c = kW == kPaired ? (j >> 2) * 16 + wn * 8 + 2 * (j & 3) + (g >> 1) : wn * 16 + 2 * j + (g >> 1);
    *reinterpret_cast<uint2*>(smem + R * 512 + ((c ^ (R & 31)) << 4) + 8 * (g & 1)) =
        make_uint2(T::pack2(v0, v1), T::pack2(v2, v3));
  }
  template <class Store>
  __device__ __forceinline__ void flush16(Store store8) const {
    __syncthreads();
    const int c = lane & 31;
#pragma unroll 4
    for (int u = 0; u < 32; ++u) {
      const int R = wave * 64 + 2 * u + (lane >> 5);
      store8(R, c, *reinterpret_cast<const uint4*>(smem + R * 512 + ((c ^ (R & 31)) << 4)));
    }
  }
  template <class Store>
  __device__ __forceinline__ void store_rows16(const f32x4 (&acc)[8][8], Store store8) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) put16(i, j, acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
    flush16(store8);
  }
  // The split's fp32 tile into part + z M cols; store column of (i, j), counted
  // from a.first, as run() says (kPaired: G at c, U at cols / 2 + c).
  __device__ __forceinline__ void store_part(const f32x4 (&acc)[8][8], int64_t cols) const {
    const int64_t c0 = this->c0 - a.first;
    const Rsrc rp = make_rsrc(a.part + (static_cast<int64_t>(blockIdx.z) * a.M + m0) * cols + c0,
                              ((a.M - m0) * cols - c0) * 4);
    const int64_t last = kW == kPaired ? cols / 2 : cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = wm * 128 + 16 * i + q;
      const bool row_ok = m0 + row < a.M;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = (kW == kPaired ? wn * 64 + 16 * (j & 3) : wn * 128 + 16 * j) + 4 * g;
        const int64_t at = kW == kPaired && j >= 4 ? cols / 2 + col : col;
        const uint32_t voff = row_ok && c0 + col < last ? static_cast<uint32_t>((row * cols + at) * 4) : kMasked;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), rp, voff, 0, 0);
      }
    }
  }
};

}  // namespace

}  // namespace qn
