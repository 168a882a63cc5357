// The building blocks of the large-M GEMM kernels (gemm_big.hip describes them):
// operand staging, the tile's reduction stages, the LoRA extension and the
// 16-bit or split store.  Shared by the kernels whose epilogues differ.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace qn {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBM = 256;
constexpr int kBN = 256;
constexpr int kBK = 64;
constexpr int kThreads = 256;
constexpr int kTileBytes = 256 * 128;
constexpr int kTabBytes = 256 * 32;
constexpr int kOffA = 0;                           // 2 stages of activation tiles
constexpr int kOffB = 2 * kTileBytes;              // 2 stages of weight tiles
constexpr int kOffT = 4 * kTileBytes;              // 2 stages of block tables
constexpr int kOffQ = kOffT + 2 * kTabBytes;       // fl32(q/127) table
constexpr int kLdsBytes = kOffQ + 256 * 4;

__device__ __forceinline__ int swz(int row) { return (row ^ (row >> 3)) & 7; }
__device__ __forceinline__ int lds_off(int row, int chunk) { return row * 128 + ((chunk ^ swz(row)) << 4); }


struct BigArgs {
  const uint16_t* act;     // X (forward) or G (backward): rows m, reduction contiguous
  int64_t act_ld;          // K (forward) or N (backward)
  NF4View W;
  const uint16_t* ext_a;   // Z (forward) or dZ (backward), M x r bf16
  const uint16_t* ext_b;   // (c B)ᵀ in bf16 (forward, N x r) or A (backward, K x r)
  uint16_t* out;           // Y (M x N) or dX (M x K)
  int64_t M, K, N, r;
  const uint16_t* wdense;  // dense path: Ŵᵀ (N x K, forward) or Ŵ (K x N, backward), bf16
  // Forward over the concatenated columns of a group of linears sharing X:
  // ext_a is then M x (ngroups r) (row stride ext_a_ld) and output columns
  // c >= gend[i] (member i+1 onwards) take their Z from column block i+1.
  // Zero / unset: one linear, ext_a row stride r.
  int64_t ext_a_ld;
  int ngroups;
  int64_t gend[kMaxGroupMembers];
  // Split-K (part non-null): workgroup z reduces elements [z k_per,
  // (z+1) k_per) and writes its fp32 tile to part + z M cols (row-major);
  // only z = 0 adds the LoRA extension.  The sum over z in order then gives
  // the output.
  float* part;
  int64_t k_per;
};

// Reduction stages [beg, end) of this workgroup.
template <bool kSplit>
__device__ __forceinline__ void stage_range(const BigArgs& a, int64_t red, int64_t step, int64_t& beg, int64_t& end) {
  const int64_t all = (red + step - 1) / step;
  beg = 0;
  end = all;
  if (kSplit) {
    beg = static_cast<int64_t>(blockIdx.z) * (a.k_per / step);
    end = beg + a.k_per / step < all ? beg + a.k_per / step : all;
  }
}

#ifndef QN_TILE_GROUP
#define QN_TILE_GROUP 4
#endif
constexpr int64_t kGroup = QN_TILE_GROUP;

// Workgroup -> output tile origin.  Workgroups are dealt to the 8 XCDs
// round-robin (id % 8); XCD x takes the x-th contiguous run of tile numbers,
// and tile numbers walk groups of kGroup row-tiles column by column, so the
// tiles of one XCD form a compact block whose activation rows and weight
// columns are shared in that XCD's L2.  A bijection for any grid.
template <int kCols = kBN>
__device__ __forceinline__ void tile_origin(int64_t& m0, int64_t& c0) {
  const int64_t ntx = gridDim.x, nty = gridDim.y, total = ntx * nty;
  const int64_t id = static_cast<int64_t>(blockIdx.y) * ntx + blockIdx.x;
  const int64_t t = (total % 8 == 0) ? (id % 8) * (total / 8) + id / 8 : id;
  const int64_t g = t / (kGroup * ntx), first = g * kGroup;
  const int64_t gm = nty - first < kGroup ? nty - first : kGroup;
  const int64_t w = t - g * kGroup * ntx;
  m0 = (first + w % gm) * kBM;
  c0 = (w / gm) * kCols;
}

// Registers carried from the load of a stage to its decode.
struct WRegs {
  uint32_t w[8];
  int q;
  float s2;
};

__device__ __forceinline__ uint32_t nib(uint32_t w, int t) { return (w >> (8 * (t >> 1) + ((t & 1) ? 0 : 4))) & 15u; }


__device__ __forceinline__ uint32_t ld32s(Rsrc r, uint32_t voff, uint32_t soff) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
}
__device__ __forceinline__ uint4 ld128s(Rsrc r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

template <class T, bool kForward, bool kKTail>
struct Big {
  const BigArgs& a;
  char* smem;
  int t, lane, wave;            // wave is wave-uniform (scalar)
  int64_t m0, c0, red;
  Rsrc r_act, r_codes, r_q, r_s2;
  float off;
  bool single;   // state without a second level: â = absmax[block]
  int s_shift;   // flat weight index -> index of its stored scale
  uint32_t act_voff[8];         // byte offset of this lane's activation chunk, stage 0
  int act_lim[8];               // forward tail: chunk valid while k0 < act_lim
  uint32_t w_voff[8];           // forward: code word of row i at stage 0; backward: [0] = row start
  uint32_t q_voff;              // second-level code of this thread's table at stage 0
  int64_t tab_e0;               // flat weight index of this thread's table block at stage 0
  int tab_row, tab_blk;
  bool tab_ok;

  __device__ Big(const BigArgs& args, char* s) : a(args), smem(s) {
    t = threadIdx.x;
    lane = t & 63;
    wave = __builtin_amdgcn_readfirstlane(t >> 6);
    tile_origin(m0, c0);
    red = kForward ? a.K : a.N;
    const int64_t P = a.K * a.N;
    r_act = make_rsrc(a.act, a.M * a.act_ld * 2);
    r_codes = make_rsrc(a.W.codes, (P + 1) / 2);
    single = a.W.absmax != nullptr;
    r_q = make_rsrc(a.W.qabsmax, single ? 0 : (P + 63) / 64);
    r_s2 = single ? make_rsrc(a.W.absmax, ((P + 63) / 64) * 4) : make_rsrc(a.W.absmax2, ((P + 16383) / 16384) * 4);
    s_shift = single ? 6 : 14;
    off = single ? 0.0f : a.W.offset[0];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // row = wave*64 + 8j + lane/8, whose swizzle is (lane/8) ^ j
      const int chunk = (lane & 7) ^ (lane >> 3) ^ j;
      const int64_t m = m0 + wave * 64 + 8 * j + (lane >> 3);
      act_voff[j] = m < a.M ? static_cast<uint32_t>((m * a.act_ld + 8 * chunk) * 2) : kMasked;
      act_lim[j] = static_cast<int>(red - 8 * chunk);
    }
    if (kForward) {
      const int rg = t >> 5, cg = t & 31;
      const int64_t col = c0 + 8 * cg;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w_voff[i] = col < a.N ? static_cast<uint32_t>(((8 * rg + i) * a.N + col) >> 1) : kMasked;
      tab_row = 8 * rg + (cg & 7);
      tab_blk = cg >> 3;
      tab_ok = c0 + 64 * tab_blk < a.N;
      tab_e0 = tab_row * a.N + c0 + 64 * tab_blk;
    } else {
      const int64_t k = c0 + t;
      w_voff[0] = k < a.K ? static_cast<uint32_t>((k * a.N) >> 1) : kMasked;
      tab_row = t;
      tab_blk = 0;
      tab_ok = k < a.K;
      tab_e0 = k * a.N;
    }
    q_voff = tab_ok ? static_cast<uint32_t>(tab_e0 >> 6) : kMasked;
  }

  __device__ char* sA(int b) const { return smem + kOffA + b * kTileBytes; }
  __device__ char* sB(int b) const { return smem + kOffB + b * kTileBytes; }
  __device__ uint16_t* tabs(int b) const { return reinterpret_cast<uint16_t*>(smem + kOffT + b * kTabBytes); }
  __device__ const float* q2t() const { return reinterpret_cast<const float*>(smem + kOffQ); }

  // Activation stage s -> LDS buffer b, straight from global memory.
  __device__ void copy_act(int64_t s, int b) const {
    const int64_t k0 = s * kBK;
    const uint32_t soff = static_cast<uint32_t>(k0 * 2);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t v = k0 < act_lim[j] ? act_voff[j] : kMasked;
      char* dst = sA(b) + (wave * 64 + 8 * j) * 128;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r_act, (lds_ptr_t)(dst), 16, v, soff, 0, 0);
    }
  }

  // Code words and the table's second-level code / scale of stage s.
  __device__ void load_w(WRegs& R, int64_t s) const {
    const int64_t k0 = s * kBK;
    if (kForward) {
      const uint32_t soff = static_cast<uint32_t>((k0 * a.N) >> 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool ok = kKTail ? k0 + 8 * (t >> 5) + i < a.K : k0 < a.K;
        R.w[i] = ld32s(r_codes, ok ? w_voff[i] : kMasked, soff);
      }
      R.q = static_cast<int>(static_cast<int8_t>(__builtin_amdgcn_raw_buffer_load_b8(
          r_q, k0 + tab_row < a.K ? q_voff : kMasked, static_cast<uint32_t>((k0 * a.N) >> 6), 0)));
      const int64_t e = tab_e0 + k0 * a.N;
      R.s2 = ld_f32(r_s2, tab_ok ? static_cast<uint32_t>((e >> s_shift) * 4) : kMasked);
    } else {
      const uint32_t soff = static_cast<uint32_t>(k0 >> 1);
      const uint32_t wv = k0 < a.N ? w_voff[0] : kMasked;
      const uint4 lo = ld128s(r_codes, wv, soff);
      const uint4 hi = ld128s(r_codes, wv, soff + 16);
      R.w[0] = lo.x; R.w[1] = lo.y; R.w[2] = lo.z; R.w[3] = lo.w;
      R.w[4] = hi.x; R.w[5] = hi.y; R.w[6] = hi.z; R.w[7] = hi.w;
      R.q = static_cast<int>(static_cast<int8_t>(
          __builtin_amdgcn_raw_buffer_load_b8(r_q, k0 < a.N ? q_voff : kMasked, static_cast<uint32_t>(k0 >> 6), 0)));
      const int64_t e = tab_e0 + k0;
      R.s2 = ld_f32(r_s2, tab_ok ? static_cast<uint32_t>((e >> s_shift) * 4) : kMasked);
    }
  }

  // Build this thread's table for stage s into table buffer b.
  __device__ void build_table(const WRegs& R, int64_t s, int b) const {
    const int64_t krow = kForward ? s * kBK + tab_row : c0 + tab_row;
    float ahat = single ? R.s2 : __fadd_rn(__fmul_rn(q2t()[R.q + 128], R.s2), off);
    if (krow >= a.K) ahat = 0.0f;   // rows past K decode to zero
    write_block_table<T>(tabs(b) + (kForward ? (tab_row * 4 + tab_blk) : tab_row) * 16, ahat);
  }

  // Split code words into byte-wise doubled nibbles: ix[2c] holds 2*code of
  // the even (high-nibble) elements of word c in its 4 bytes, ix[2c+1] those
  // of the odd (low-nibble) elements, so a lookup address is table + 1 byte.
  __device__ void split_codes(const WRegs& R, uint32_t (&ix)[16]) const {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ix[2 * c] = (R.w[c] >> 3) & 0x1E1E1E1Eu;
      ix[2 * c + 1] = (R.w[c] << 1) & 0x1E1E1E1Eu;
    }
  }

  // Decode part `part` (0..7) of this thread's share of a stage into weight
  // buffer b: forward column `part` of the thread's 8 columns (8 rows, one
  // table each); backward chunk `part` of its row (8 elements, one table).
  __device__ void decode_part(const uint32_t (&ix)[16], int b, int part) const {
    const char* tb = reinterpret_cast<const char*>(tabs(b));
    char* dst = sB(b);
    uint32_t d[4];
    if (kForward) {
      const int rg = t >> 5, cg = t & 31;
      const char* trow = tb + ((8 * rg) * 4 + (cg >> 3)) * 32;   // table of row 8rg + i at trow + 128 i
      const int sh = 8 * (part >> 1);
      const int odd = part & 1;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t i0 = (ix[2 * (2 * p) + odd] >> sh) & 0xFFu;
        const uint32_t i1 = (ix[2 * (2 * p + 1) + odd] >> sh) & 0xFFu;
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(trow + (2 * p) * 128 + i0);
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(trow + (2 * p + 1) * 128 + i1);
        d[p] = lo | (hi << 16);
      }
      *reinterpret_cast<uint4*>(dst + lds_off(8 * cg + part, rg)) = make_uint4(d[0], d[1], d[2], d[3]);
    } else {
      const char* tr = tb + tab_row * 32;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        // elements 2p (high nibble of byte p) and 2p+1 (low nibble)
        const uint32_t i0 = (ix[2 * part] >> (8 * p)) & 0xFFu;
        const uint32_t i1 = (ix[2 * part + 1] >> (8 * p)) & 0xFFu;
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(tr + i0);
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(tr + i1);
        d[p] = lo | (hi << 16);
      }
      *reinterpret_cast<uint4*>(dst + lds_off(t, part)) = make_uint4(d[0], d[1], d[2], d[3]);
    }
  }

  // One stage of MFMAs from buffer b: 4 substeps of 16 reduction elements,
  // each 4 activation x 4 weight fragments (32 rows x 16 values; lane l holds
  // row l%32, values 8*(l/32)..+7) and 16 v_mfma_f32_32x32x16_bf16.
  struct Frags {
    typename T::v8 a[4], w[4];
  };
  __device__ void load_frags(int b, int ks, Frags& F) const {
    const int r32 = lane & 31, h = lane >> 5, wm = wave >> 1, wn = wave & 1;
    const char* A = sA(b);
    const char* Bt = sB(b);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      F.a[i] = *reinterpret_cast<const typename T::v8*>(A + lds_off(wm * 128 + 32 * i + r32, 2 * ks + h));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      F.w[j] = *reinterpret_cast<const typename T::v8*>(Bt + lds_off(wn * 128 + 32 * j + r32, 2 * ks + h));
  }
  __device__ static void mma(const Frags& F, f32x16 (&acc)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = T::mfma32(F.w[j], F.a[i], acc[i][j]);
  }
  __device__ void compute(int b, f32x16 (&acc)[4][4]) const {
    Frags F;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      load_frags(b, ks, F);
      mma(F, acc);
    }
  }
};

// Dense core: both operands are 16-bit matrices with the reduction
// contiguous (activations M x red and the dequantized weight, rows x red).
// 64-element stages go through three LDS slots of 256 activation rows and two
// of 256 weight rows, 128 bytes a row in the fused kernel's layout (chunk c of
// row R at c ^ ((R ^ R >> 3) & 7)): the whole 160 KB.  Copies are buffer loads
// straight into LDS, each instruction 8 rows x 128 bytes, i.e. whole cache
// lines: issuing the same bytes as 16 half-line rows per instruction cost about
// 10% more time.  In stage u a wave copies its share of the activations of
// stage u+2 during the first substep (they have 1.75 stages to land) and of its
// weights during the last (0.75 of a stage), one copy per two MFMAs (in bursts
// they fill the TA command FIFO and stall the MFMA stream); the one barrier per
// stage sits before the last substep, whose fragments are already in registers,
// and waits for all but the activations of stage u+2.
constexpr int kDenseW = 3 * kTileBytes;     // the two weight slots follow the three activation slots
constexpr int kDenseLds = 5 * kTileBytes;   // 160 KB

template <class T, bool kForward, bool kKTail>
struct Dense {
  const BigArgs& a;
  char* smem;
  int t, lane, wave;
  int64_t m0, c0, red;
  Rsrc r_act, r_w;
  uint32_t act_voff[8], w_voff[8];   // copy j: row wave*64 + 8j + lane/8, chunk (lane&7)^(lane>>3)^j
  int lim[8];                        // reduction tail: copy j's chunk valid while k0 < lim[j]
  int fA[4], fW[4];                  // fragment offsets within a slot at substep 0
  // Stages: n_main of the product (from s_beg), then the LoRA extension's
  // ceil(r_ext / 64) over (Z, (c B)ᵀ) or (dZ, A), copied like the others.
  int64_t s_beg, n_main, r_ext, lda, cols;
  Rsrc r_ea, r_eb;

  __device__ Dense(const BigArgs& args, char* s) : a(args), smem(s) {
    t = threadIdx.x;
    lane = t & 63;
    wave = __builtin_amdgcn_readfirstlane(t >> 6);
    tile_origin(m0, c0);
    red = kForward ? a.K : a.N;
    const int64_t wrows = kForward ? a.N : a.K;
    cols = wrows;
    r_act = make_rsrc(a.act, a.M * red * 2);
    r_w = make_rsrc(a.wdense, wrows * red * 2);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // row = wave*64 + 8j + lane/8, whose swizzle is (lane/8) ^ j
      const int chunk = (lane & 7) ^ (lane >> 3) ^ j;
      const int row = wave * 64 + 8 * j + (lane >> 3);
      const int64_t m = m0 + row, n = c0 + row;
      act_voff[j] = m < a.M ? static_cast<uint32_t>((m * red + 8 * chunk) * 2) : kMasked;
      w_voff[j] = n < wrows ? static_cast<uint32_t>((n * red + 8 * chunk) * 2) : kMasked;
      lim[j] = static_cast<int>(red - 8 * chunk);
    }
    const int r32 = lane & 31, h = lane >> 5, wm = wave >> 1, wn = wave & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fA[i] = lds_off(wm * 128 + 32 * i + r32, h);
      fW[i] = kDenseW + lds_off(wn * 128 + 32 * i + r32, h);
    }
    lda = a.ext_a_ld ? a.ext_a_ld : a.r;
    int64_t zoff = 0;   // grouped forward: this tile's member's block of Z columns
    if (kForward)
      for (int i = 0; i < a.ngroups; ++i) zoff += c0 >= a.gend[i] ? a.r : 0;
    r_ea = make_rsrc(a.ext_a + zoff, (a.M * lda - zoff) * 2);
    r_eb = make_rsrc(a.ext_b, cols * a.r * 2);
  }
  // this workgroup's stages (with_ext: it also adds the LoRA extension)
  __device__ int64_t set_stages(int64_t beg, int64_t end, bool with_ext) {
    s_beg = beg;
    n_main = end - beg;
    r_ext = with_ext ? a.r : 0;
    return n_main + (r_ext + kBK - 1) / kBK;
  }

  // slot 0 in the fused kernel's names, for the LoRA extension after the loop
  __device__ char* sA(int) const { return smem; }
  __device__ char* sB(int) const { return smem + kTileBytes; }

  // Copy of rows wave*64 + 8j .. +7 of stage u (counted from s_beg), of the
  // activations (kW false) or the weight, to byte `slot` of LDS.  Past the
  // reduction end and the extension: masked.  kMix: u may be an extension
  // stage (else u < n_main, known to the caller).
  template <bool kMix, bool kW>
  __device__ void copy_one(int64_t u, int slot, int j) const {
    char* dst = smem + slot + (wave * 64 + 8 * j) * 128;
    if (!kMix || u < n_main) {
      const int64_t k0 = (s_beg + u) * kBK;
      const uint32_t soff = static_cast<uint32_t>(k0 * 2);
      const bool ok = kKTail ? k0 < lim[j] : k0 < red;
      if (!kW)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r_act, (lds_ptr_t)(dst), 16, ok ? act_voff[j] : kMasked, soff, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r_w, (lds_ptr_t)(dst), 16, ok ? w_voff[j] : kMasked, soff, 0, 0);
    } else {
      const int row = wave * 64 + 8 * j + (lane >> 3);
      const int64_t e = (u - n_main) * kBK + 8 * ((lane & 7) ^ (lane >> 3) ^ j);
      if (!kW) {
        const int64_t m = m0 + row;
        const uint32_t v = (m < a.M && e < r_ext) ? static_cast<uint32_t>((m * lda + e) * 2) : kMasked;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r_ea, (lds_ptr_t)(dst), 16, v, 0, 0, 0);
      } else {
        const int64_t n = c0 + row;
        const uint32_t v = (n < cols && e < r_ext) ? static_cast<uint32_t>((n * a.r + e) * 2) : kMasked;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r_eb, (lds_ptr_t)(dst), 16, v, 0, 0, 0);
      }
    }
  }

  struct Frags {
    typename T::v8 a[4], w[4];
  };
  // Fragment q (activation q/2 for even q, weight q/2 for odd q) of
  // substep ks of the slots at bytes sa and sw: chunk 2ks + h of its row, i.e.
  // the substep-0 offset with bits 5-6 flipped by ks (fW holds kDenseW).
  __device__ void read_one(int sa, int sw, int ks, int q, Frags& F) const {
    if ((q & 1) == 0)
      F.a[q >> 1] = *reinterpret_cast<const typename T::v8*>(smem + sa + (fA[q >> 1] ^ (ks << 5)));
    else
      F.w[q >> 1] = *reinterpret_cast<const typename T::v8*>(smem + sw + (fW[q >> 1] ^ (ks << 5)));
  }
  __device__ void load_frags(int sa, int sw, int ks, Frags& F) const {
#pragma unroll
    for (int q = 0; q < 8; ++q) read_one(sa, sw, ks, q, F);
  }

  // 16 MFMAs from Fc; in their shadow the 8 reads of substep ksn of the slots
  // sa and sw into Fn (within the first 8 MFMAs, so the last 8 cover their
  // latency) and, after every second one, copy g of `side`.  The order is
  // pinned with scheduling barriers.
  template <class Side>
  __device__ void sub_step(const Frags& Fc, Frags& Fn, int sa, int sw, int ksn, f32x16 (&acc)[4][4], Side side) const {
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      acc[m >> 2][m & 3] = T::mfma32(Fc.w[m & 3], Fc.a[m >> 2], acc[m >> 2][m & 3]);
      __builtin_amdgcn_sched_barrier(0);
      if (m < 8) {
        read_one(sa, sw, ksn, m, Fn);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (m & 1) {
        side(m >> 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // Stage u from activation slot sa and weight slot sw (bytes), the next stage's
  // in sa1 and sw1; stage u+2 goes to sa2 and sw (see dense_loop).
  template <bool kMix>
  __device__ void stage(int64_t u, int sa, int sa1, int sa2, int sw, int sw1, Frags& F0, Frags& F1,
                        f32x16 (&acc)[4][4]) const {
    sub_step(F0, F1, sa, sw, 1, acc, [&](int g) { copy_one<kMix, false>(u + 2, sa2, g); });
    sub_step(F1, F0, sa, sw, 2, acc, [](int) {});
    sub_step(F0, F1, sa, sw, 3, acc, [](int) {});
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    sub_step(F1, F0, sa1, sw1, 0, acc, [&](int g) { copy_one<kMix, true>(u + 2, kDenseW + sw, g); });
  }

  // finish() is called without the extension (it ran as the last stages).
  __device__ void compute(int, f32x16 (&)[4][4]) const {}
};

// The dense core's loop over this workgroup's stages (kSplit: blockIdx.z's
// share of the reduction): clears and fills acc, and releases LDS.
// Stage u (counted from the first of this workgroup's range; the LoRA
// extension's stages follow the product's) has its activations in slot u % 3
// and its weights in slot u % 2.  The barrier of stage u, before its last
// substep, says: every wave has read all of stage u (its last substep's
// fragments are in registers) and stage u+1 has landed.  The weights of stage
// u+2 follow it into slot u % 2; the activations of stage u+2 went into slot
// (u - 1) % 3, free since the barrier before.  Copies past the end are masked
// or land in a slot that is never read.
template <bool kSplit, class Core>
__device__ __forceinline__ void dense_loop(Core& k, const BigArgs& a, f32x16 (&acc)[4][4]) {
  int64_t s_beg, s_end;
  stage_range<kSplit>(a, k.red, kBK, s_beg, s_end);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int64_t total = k.set_stages(s_beg, s_end, !kSplit || blockIdx.z == 0);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    k.template copy_one<true, false>(0, 0, j);
    k.template copy_one<true, true>(0, kDenseW, j);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) k.template copy_one<true, false>(1, kTileBytes, j);
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 0));
  __builtin_amdgcn_s_barrier();
  typename Core::Frags F0, F1;
  k.load_frags(0, 0, 0, F0);
#pragma unroll
  for (int j = 0; j < 8; ++j) k.template copy_one<true, true>(1, kDenseW + kTileBytes, j);
  int sa = 0, sa1 = kTileBytes, sa2 = 2 * kTileBytes, sw = 0;
  auto turn = [&] {
    const int s = sa;
    sa = sa1;
    sa1 = sa2;
    sa2 = s;
    sw ^= kTileBytes;
  };
  int64_t u = 0;
  // stages whose copies (of u+2) are all of the product, then the rest
  for (; u + 2 < k.n_main; ++u, turn()) k.template stage<false>(u, sa, sa1, sa2, sw, sw ^ kTileBytes, F0, F1, acc);
  for (; u < total; ++u, turn()) k.template stage<true>(u, sa, sa1, sa2, sw, sw ^ kTileBytes, F0, F1, acc);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
}

// LoRA extension: r more reduction steps over (Z, (c B)ᵀ) in the forward or
// (dZ, A) in the backward; both operands are row-major with r contiguous
// (M x r and cols x r), staged into the 64-wide LDS layout of the main loop.
// Then the bf16 store: the tile goes through LDS (row-major, 512 bytes per
// row, 16-byte chunk q of row R at q ^ (R & 31)) so that every global store
// writes whole 512-byte row segments.  Shared by the fused and dense kernels;
// the main loop has released LDS when this starts.
template <class T, bool kForward, bool kSplit, bool kExt, class Core>
__device__ __forceinline__ void finish(const Core& k, const BigArgs& a, f32x16 (&acc)[4][4]) {
  const int lane = k.lane, t = k.t;
  const int64_t cols = kForward ? a.N : a.K;
  const int64_t lda = a.ext_a_ld ? a.ext_a_ld : a.r;
  int64_t zoff = 0;   // grouped forward: this tile's member's block of Z columns
  if (kForward)
    for (int i = 0; i < a.ngroups; ++i) zoff += k.c0 >= a.gend[i] ? a.r : 0;
  const Rsrc re = make_rsrc(a.ext_a + zoff, (a.M * lda - zoff) * 2);
  const Rsrc rb = make_rsrc(a.ext_b, cols * a.r * 2);
  const int64_t r_ext = kExt && (!kSplit || blockIdx.z == 0) ? a.r : 0;
  for (int64_t j0 = 0; j0 < r_ext; j0 += kBK) {
    const int c = t & 7;
    const int64_t j = j0 + 8 * c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = (t >> 3) + 32 * i;
      const int64_t m = k.m0 + row, n = k.c0 + row;
      const uint4 v = ld_b128(re, (m < a.M && j < a.r) ? static_cast<uint32_t>((m * lda + j) * 2) : kMasked);
      const uint4 w = ld_b128(rb, (n < cols && j < a.r) ? static_cast<uint32_t>((n * a.r + j) * 2) : kMasked);
      *reinterpret_cast<uint4*>(k.sA(0) + lds_off(row, c)) = v;
      *reinterpret_cast<uint4*>(k.sB(0) + lds_off(row, c)) = w;
    }
    __syncthreads();
    k.compute(0, acc);
    __syncthreads();
  }

  // Lane l holds, for tile (i, j), output row 32i + l%32 and, for each jj,
  // the 4 columns 32j + 8jj + 4(l/32) .. +3.
  if constexpr (kSplit) {
    // split-K: the fp32 tile, 16 bytes per buffer store; rows past M and
    // columns past cols (cols % 8 == 0) are masked.
    const int r32 = lane & 31, h = lane >> 5, wm = k.wave >> 1, wn = k.wave & 1;
    const Rsrc rp = make_rsrc(a.part + (static_cast<int64_t>(blockIdx.z) * a.M + k.m0) * cols + k.c0,
                              ((a.M - k.m0) * cols - k.c0) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = wm * 128 + 32 * i + r32;
      const bool row_ok = k.m0 + row < a.M;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int col = wn * 128 + 32 * j + 8 * jj + 4 * h;
          const uint32_t voff =
              (row_ok && k.c0 + col < cols) ? static_cast<uint32_t>((row * cols + col) * 4) : kMasked;
          const f32x4 v = {acc[i][j][4 * jj], acc[i][j][4 * jj + 1], acc[i][j][4 * jj + 2], acc[i][j][4 * jj + 3]};
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rp, voff, 0, 0);
        }
    }
    return;
  }
  char* st = k.sA(0);
  {
    const int r32 = lane & 31, h = lane >> 5, wm = k.wave >> 1, wn = k.wave & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int R = wm * 128 + 32 * i + r32;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int q = wn * 16 + 4 * j + jj;
          uint2 v;
          v.x = T::pack2(acc[i][j][4 * jj], acc[i][j][4 * jj + 1]);
          v.y = T::pack2(acc[i][j][4 * jj + 2], acc[i][j][4 * jj + 3]);
          *reinterpret_cast<uint2*>(st + R * 512 + ((q ^ r32) << 4) + 8 * h) = v;
        }
    }
  }
  __syncthreads();
  {
    const int q = lane & 31;
    const int64_t n = k.c0 + 8 * q;
#pragma unroll 4
    for (int u = 0; u < 32; ++u) {
      const int R = k.wave * 64 + 2 * u + (lane >> 5);
      const int64_t m = k.m0 + R;
      const uint4 v = *reinterpret_cast<const uint4*>(st + R * 512 + ((q ^ (R & 31)) << 4));
      // non-temporal: the output streams out during the epilogue instead of
      // waiting, dirty in L2, for the end-of-kernel release (1-2 us per launch)
      if (m < a.M && n < cols)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(a.out + m * cols + n));
    }
  }
}

}  // namespace

}  // namespace qn
