// Softmax cross entropy of the frozen output head, with its gradient, for
// gfx950: logits s = X Wᵀ (M x V, never kept), per row
//   loss = w (lse - s_t),  lse = log sum_v e^{s_v},  dX = w sum_v (p_v - [v = t]) W_v.
//
// One pass over the vocabulary in pieces of at most kPieceBytes of 16-bit
// probabilities; 2 M K V operations for the loss and as many for dX.  Per piece:
//   1. head_logits_kernel: the GEMM of X and the piece's rows of W.  Its
//      epilogue turns a tile's logits into powers of two relative to an integer
//      bound of their own row and 128 columns, P = 2^(s log2 e - ref), ref = 0 or
//      the ceil of the largest (head_ref): P (16 bits, one rounding), ref and the
//      sum of the unrounded P go to memory.  The target's own column is left out of all
//      three; its logit is kept in fp32.  (P is an operand of the next product's
//      MFMAs, hence 16 bits; each term of dX carries that one rounding, the loss
//      and lse none.)
//   2. head_rows_kernel: per row the running bound and sum over the pieces, and
//      P times 2^(ref - bound) where they differ: a power of two, so no second
//      rounding - but for fp16 values that fall below 2^-28 of the row's bound,
//      which become subnormal and are off by at most 2^-39 of it.
//   3. head_dx_kernel: the GEMM of P and the same rows of W, read in their
//      stored order and turned in registers on the way into LDS, added to the
//      earlier pieces' fp32 sums times 2^(old bound - bound).
// With l the sum without the target and u = log l + bound - s_t, the row's loss
// is w softplus(u), 1 - p_t = sigmoid(u) =: g and
//   dX = w g (sum_{v != t} P_v W_v / l - W_t),
// so that neither the loss nor the target's part of dX suffers from
// cancellation where the target is nearly certain.
// Bound by the matrix cores; with few rows by the read of W.  Measured at 4096
// rows of 4096 columns and 32000 entries: 1665 us (1.29 PFLOP/s), of it the
// logits 798 to 870 (MFMA pipes 66 % busy at 1.78 GHz), the gradient product 840 to
// 928 (58 % at 1.84 GHz), the rows 12 (90 where the groups' bounds differ and P is
// rescaled).
#include <hip/hip_ext.h>

#include "gemm16.hpp"

namespace qn {

namespace {

constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;
#ifndef QN_HEAD_PIECE_MB
#define QN_HEAD_PIECE_MB 256
#endif
constexpr int64_t kPieceBytes = static_cast<int64_t>(QN_HEAD_PIECE_MB) << 20;

// P is stored times 2^kShift: fp16 has few exponents, and its small values would
// lose bits below 2^-14.
template <class T>
constexpr int head_shift() { return T::kDtype == F16::kDtype ? 14 : 0; }

// The bound of a row's 128 columns with largest logit `top`.  bf16 has fp32's
// exponents, so within 2^-64 .. 2^40 the logits stand as they are (bound 0): a
// row whose groups all do, as a language model's, needs no common bound made for
// it afterwards.  A group's terms below 2^-126 are then 2^-62 of its largest.
template <class T>
__device__ __forceinline__ float head_ref(float top) {
  // nothing but masked columns: any bound serves, every P is 0
  if (top == -__builtin_inff()) return 0.0f;
  const float e = __builtin_ceilf(top * kLog2e);
  return T::kDtype == Bf16::kDtype && e >= -64.0f && e <= 40.0f ? 0.0f : e;
}

struct HeadArgs {
  const int64_t* targets;
  int64_t v0, nv, ldp;       // this piece's first vocabulary row, its rows, P's row stride
  int64_t V, ignore;
  uint16_t* P;               // M x ldp, or null: the loss alone
  float2* stats;             // M x nh: (bound, sum) of each 128 columns
  int64_t nh;
  float* st;                 // M: the target's logit
};

template <class T, bool kStore>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void head_logits_kernel(G16Args a,
                                                                                                         HeadArgs p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Core16<T, kRows> k(a, smem);
  f32x4 acc[8][8];
  k.template run<false>(acc);
  // a row's 128 columns of this wave: 32 in each of the four lanes q, q + 16, q + 32, q + 48
  const int64_t cbase = k.c0 + k.wn * 128;         // this wave's first column of the piece
  const int64_t half = cbase >> 7;
  const bool ragged = cbase + 128 > p.nv;          // the wave has columns past the piece
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t m = k.m0 + k.wm * 128 + 16 * i + k.q;
    const int64_t t = m < a.M ? p.targets[m] : -1;
    const int64_t d = t - p.v0 - cbase;
    // the target, if it is one of this wave's columns (an ignored row has none)
    const bool here = t >= 0 && t < p.V && t != p.ignore && d >= 0 && d < 128;
    float v[32];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[4 * j + e] = acc[i][j][e];
        asm("" : "+v"(v[4 * j + e]));   // (values that the branches below change would stay accumulators)
      }
    if (ragged) {
      const int left = static_cast<int>(p.nv - cbase) - 4 * k.g;
#pragma unroll
      for (int x = 0; x < 32; ++x) v[x] = 16 * (x >> 2) + (x & 3) < left ? v[x] : -__builtin_inff();
    }
    // column 16 j + 4 g + e of a row is value 4 j + e of its lane g
    const bool mine = here && ((d >> 2) & 3) == k.g;
    if (__any(mine)) {
      const int own = mine ? static_cast<int>((d >> 4) * 4 + (d & 3)) : -1;
      float s = 0.0f;
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        s = own == x ? v[x] : s;
        v[x] = own == x ? -__builtin_inff() : v[x];
      }
      if (mine) p.st[m] = s;
    }
    float top = v[0];
#pragma unroll
    for (int x = 1; x < 32; ++x) top = fmaxf(top, v[x]);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float ref = head_ref<T>(top);
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < 32; ++x) {
      v[x] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[x], kLog2e, -ref));
      sum += v[x];
      v[x] *= static_cast<float>(1 << head_shift<T>());
    }
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if (k.g == 0 && m < a.M && half < p.nh) p.stats[m * p.nh + half] = make_float2(ref, sum);
    if constexpr (kStore) {
#pragma unroll
      for (int j = 0; j < 8; ++j) k.put16(i, j, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
  }
  if constexpr (kStore) {
    k.flush16([&](int R, int c, const uint4& x) {
      const int64_t m = k.m0 + R, n = k.c0 + 8 * c;
      if (m < a.M && n < p.ldp) *reinterpret_cast<uint4*>(p.P + m * p.ldp + n) = x;
    });
  }
}

// The same with the reduction split: fp32 partials of the tiles, M x ldp a split.
template <class T>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void head_part_kernel(G16Args a,
                                                                                                       int64_t ldp) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Core16<T, kRows> k(a, smem);
  f32x4 acc[8][8];
  k.template run<true>(acc);
  k.store_part(acc, ldp);
}

// Their sums in split order, and the epilogue of head_logits_kernel: 32 lanes
// take a row's 128 columns, four each.  Up to kJoin splits are requested at once.
template <class T, bool kStore>
__global__ __launch_bounds__(256) void head_join_kernel(const float* __restrict__ part, int64_t splits, int64_t M,
                                                        HeadArgs p) {
  constexpr int kJoin = 8;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const bool live = unit < M * p.nh;
  const int64_t m = live ? unit / p.nh : 0, half = live ? unit - m * p.nh : 0;
  const int64_t col = half * 128 + 4 * lane, plane = M * p.ldp;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool stored = live && col < p.ldp;
  if (stored) {
    const float* from = part + m * p.ldp + col;
    for (int64_t z = 0; z < splits; z += kJoin) {
      f32x4 x[kJoin];
#pragma unroll
      for (int i = 0; i < kJoin; ++i)
        x[i] = z + i < splits ? *reinterpret_cast<const f32x4*>(from + (z + i) * plane) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kJoin; ++i) v += x[i];
    }
  }
  const int64_t t = live ? p.targets[m] : -1;
  const bool wanted = t >= 0 && t < p.V && t != p.ignore;
  float top = -__builtin_inff();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (wanted && stored && col + e == t - p.v0) {
      p.st[m] = v[e];
      v[e] = -__builtin_inff();
    }
    if (col + e >= p.nv) v[e] = -__builtin_inff();
    top = fmaxf(top, v[e]);
  }
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
  const float ref = head_ref<T>(top);
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[e], kLog2e, -ref));
    sum += v[e];
    v[e] *= static_cast<float>(1 << head_shift<T>());
  }
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) sum += __shfl_xor(sum, s, 64);
  if (live && lane == 0) p.stats[m * p.nh + half] = make_float2(ref, sum);
  if (kStore && stored)
    *reinterpret_cast<uint2*>(p.P + m * p.ldp + col) = make_uint2(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]));
}

struct RowArgs {
  const float2* stats;
  int64_t nh, ldp, M, V, ignore;
  uint16_t* P;               // null: the loss alone
  const float2* run_in;      // (bound, sum) of the earlier pieces; null for the first
  float2* run_out;
  const float* st;
  const int64_t* targets;
  const float* weights;      // null: 1
  float* alpha;              // 2^(old bound - bound), for the earlier pieces' dX sums
  float* loss;               // written with the last piece (else null)
  float* lse;
  float2* coef;              // last piece: (w g, 1 / l); (0, .) marks an ignored row, (NaN, .) a bad target
};

__device__ __forceinline__ float wg_max(float v, float* red) {
  for (int s = 32; s >= 1; s >>= 1) v = fmaxf(v, __shfl_xor(v, s, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  return v;
}
__device__ __forceinline__ float wg_sum(float v, float* red) {
  for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (red[0] + red[1]) + (red[2] + red[3]);
  __syncthreads();
  return v;
}

// One row and a slice of its columns (blockIdx.y); every slice forms the row's
// new bound and sum (the same bits), slice 0 writes them.
template <class T>
__global__ __launch_bounds__(256) void head_rows_kernel(RowArgs p) {
  __shared__ float red[4];
  const int64_t m = blockIdx.x;
  const int t = threadIdx.x;
  const float2* s = p.stats + m * p.nh;
  float2 old = make_float2(-__builtin_inff(), 0.0f);
  if (p.run_in != nullptr) old = p.run_in[m];
  float top = old.x, low = __builtin_inff();
  for (int64_t i = t; i < p.nh; i += 256) {
    const float2 v = s[i];
    // an empty group bounds nothing; a NaN sum must reach the row's
    if (v.y != 0.0f) {
      top = fmaxf(top, v.x);
      low = fminf(low, v.x);
    }
  }
  top = wg_max(top, red);
  low = -wg_max(-low, red);
  if (top == -__builtin_inff()) top = 0.0f;   // nothing in the row so far
  float sum = 0.0f;
  for (int64_t i = t; i < p.nh; i += 256) {
    const float2 v = s[i];
    if (v.y != 0.0f) sum += v.y * __builtin_amdgcn_exp2f(v.x - top);
  }
  sum = wg_sum(sum, red);
  const float back = old.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(old.x - top);
  sum += old.y == 0.0f ? 0.0f : old.y * back;
  if (blockIdx.y == 0 && t == 0) {
    p.run_out[m] = make_float2(sum == 0.0f ? -__builtin_inff() : top, sum);
    if (p.alpha != nullptr) p.alpha[m] = back;
    if (p.loss != nullptr) {
      const int64_t target = p.targets[m];
      const float others = sum == 0.0f ? -__builtin_inff() : (top + __builtin_log2f(sum)) * kLn2;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (target == p.ignore) {
        p.loss[m] = 0.0f;
        p.lse[m] = others;
        if (p.coef != nullptr) p.coef[m] = make_float2(0.0f, -1.0f);
      } else if (target < 0 || target >= p.V) {
        p.loss[m] = __builtin_nanf("");
        p.lse[m] = others;
        if (p.coef != nullptr) p.coef[m] = make_float2(__builtin_nanf(""), 1.0f);
      } else {
        const float w = p.weights != nullptr ? p.weights[m] : 1.0f;
        // a target logit of +inf: lse - s_t is inf - inf, a NaN, as any overflow's
        const float s = p.st[m], inf = __builtin_inff();
        const float u = s == inf ? __builtin_nanf("") : others - s;
        const float e = expf(-fabsf(u)), l1 = log1pf(e);
        const float up = fmaxf(u, 0.0f) + l1;                 // softplus(u); -inf gives 0
        const float g = (u >= 0.0f ? 1.0f : e) / (1.0f + e);  // sigmoid(u)
        p.loss[m] = w * (u != u ? u : up);
        p.lse[m] = fabsf(s) != inf ? s + (u != u ? u : up) : (s < 0.0f || others != others ? others : s);
        if (p.coef != nullptr) p.coef[m] = make_float2(w * (u != u ? u : g), inv);
      }
    }
  }
  if (p.P == nullptr || low >= top) return;   // (one bound, or nothing)
  // 128 columns (16 chunks of 8) share a factor, an exact power of two
  uint16_t* row = p.P + m * p.ldp;
  const int64_t chunks = p.ldp / 8;
  const int64_t step = static_cast<int64_t>(gridDim.y) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.y) * 256 + t; i < chunks; i += step) {
    const float2 v = s[i >> 4];
    if (v.x == top || v.y == 0.0f) continue;
    const float f = __builtin_amdgcn_exp2f(v.x - top);
    uint4 x = *reinterpret_cast<const uint4*>(row + 8 * i);
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = T::pack2(T::widen(w[c] & 0xffffu) * f, T::widen(w[c] >> 16) * f);
    *reinterpret_cast<uint4*>(row + 8 * i) = x;
  }
}

// What becomes of a piece's product at rows m and columns of dX.
struct DxArgs {
  int64_t M, K;
  const float* part;         // splits x M x K partials of a split product, else null
  int64_t splits;
  const float* prev;         // earlier pieces' sums M x K, or null
  const float* alpha;
  float* sum;                // this piece's sums (not the last piece), else null
  const float2* coef;        // last piece
  const uint16_t* W;         // V x K, for the target's row
  const int64_t* targets;
  uint16_t* dX;
  float unshift;             // 2^-shift of P
};

// Columns col + 16 j .. + 3, j < N, of row m: v[j] = this piece's product.  All
// loads of the row are requested before the first is used (one after the other,
// each waits for memory behind the stores of the last).
template <class T, int N>
__device__ __forceinline__ void dx_store(const DxArgs& p, int64_t m, int64_t col, f32x4 (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] *= p.unshift;
  if (p.prev != nullptr) {
    const float al = p.alpha[m];
    f32x4 o[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
      o[j] = col + 16 * j < p.K ? *reinterpret_cast<const f32x4*>(p.prev + m * p.K + col + 16 * j) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (al != 0.0f) v[j] += o[j] * al;   // 0: nothing was summed before
  }
  if (p.sum != nullptr) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (col + 16 * j < p.K) *reinterpret_cast<f32x4*>(p.sum + m * p.K + col + 16 * j) = v[j];
    return;
  }
  const float2 c = p.coef[m];
  const bool counts = c.x == c.x && c.y >= 0.0f;
  uint2 wt[N];
  const uint16_t* from = p.W + (counts ? p.targets[m] : 0) * p.K + col;
#pragma unroll
  for (int j = 0; j < N; ++j)
    wt[j] = counts && col + 16 * j < p.K ? *reinterpret_cast<const uint2*>(from + 16 * j) : make_uint2(0, 0);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float t[4] = {T::widen(wt[j].x & 0xffffu), T::widen(wt[j].x >> 16), T::widen(wt[j].y & 0xffffu), T::widen(wt[j].y >> 16)};
    float r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = counts ? c.x * (__builtin_fmaf(v[j][e], c.y, -t[e])) : (c.x != c.x ? c.x : 0.0f);
    if (col + 16 * j < p.K)
      *reinterpret_cast<uint2*>(p.dX + m * p.K + col + 16 * j) = make_uint2(T::pack2(r[0], r[1]), T::pack2(r[2], r[3]));
  }
}

// The sums over the splits of a piece, then the same.
template <class T>
__global__ __launch_bounds__(256) void head_sum_kernel(DxArgs p) {
  const uint32_t per = static_cast<uint32_t>(p.K / 4), count = static_cast<uint32_t>(p.M) * per;
  const int64_t plane = p.M * p.K;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < count; i += gridDim.x * 256) {
    const int64_t m = i / per, at = static_cast<int64_t>(i) * 4;
    f32x4 v = *reinterpret_cast<const f32x4*>(p.part + at);
#pragma unroll 8
    for (int64_t z = 1; z < p.splits; ++z) v += *reinterpret_cast<const f32x4*>(p.part + z * plane + at);
    f32x4 one[1] = {v};
    dx_store<T, 1>(p, m, at - m * p.K, one);
  }
}

// P (M x nv) times the piece's rows of W (nv x K).
template <class T, bool kSplit>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void head_dx_kernel(G16Args a, DxArgs p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Core16<T, kTurned> k(a, smem);
  f32x4 acc[8][8];
  k.template run<kSplit>(acc);
  if constexpr (kSplit) {
    k.store_part(acc, p.K);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t m = k.m0 + k.wm * 128 + 16 * i + k.q;
    if (m < p.M) dx_store<T, 8>(p, m, k.c0 + k.wn * 128 + 4 * k.g, acc[i]);
  }
}

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// Pieces of the vocabulary and splits of dX's reduction.
struct HeadPlan {
  int64_t pieces, rows;             // rows per piece, a multiple of 256
  int64_t splits, k_per;
  SplitPlan logits;                 // of their reduction, for a whole piece
  int64_t p_bytes, stats_bytes, row_bytes, sum_bytes, part_bytes;   // part: the logits' or dX's, one after the other
  int64_t total() const { return p_bytes + stats_bytes + 6 * row_bytes + sum_bytes + part_bytes; }
};

// A piece keeps its probabilities within kPieceBytes, its bounds and sums within
// kStatsBytes (which without dX is what M limits a piece by) and its rows of W
// within 2^29 elements (32-bit offsets).  Few tiles' reductions are split: the
// logits' over K, dX's over the piece's rows.
constexpr int64_t kStatsBytes = int64_t(64) << 20;
HeadPlan head_plan(int64_t M, int64_t K, int64_t V, bool need_dx) {
  HeadPlan h{};
  int64_t most = (int64_t(1) << 29) / K;
  if (need_dx && kPieceBytes / 2 / M < most) most = kPieceBytes / 2 / M;
  if (kStatsBytes / 8 / M * 128 < most) most = kStatsBytes / 8 / M * 128;
  most = most / 256 * 256;
  if (most < 256) most = 256;
  h.pieces = (V + most - 1) / most;
  h.rows = ((V + h.pieces - 1) / h.pieces + 255) / 256 * 256;
  h.pieces = (V + h.rows - 1) / h.rows;
  h.stats_bytes = align256(M * (h.rows / 128) * 8);
  h.row_bytes = align256(M * 8);
  h.splits = 1;
  h.k_per = h.rows;
  const int64_t width = V < h.rows ? (V + 63) / 64 * 64 : h.rows;
  h.logits = plan_split16(M, width, K);
  h.part_bytes = h.logits.part_bytes;
  if (!need_dx) return h;
  h.p_bytes = align256(M * width * 2);
  if (h.pieces > 1) h.sum_bytes = align256(M * K * 4);
  const SplitPlan dx = plan_split16(M, K, width);
  h.splits = dx.splits;
  h.k_per = dx.k_per;
  if (dx.part_bytes > h.part_bytes) h.part_bytes = dx.part_bytes;
  return h;
}

template <class T, bool kStore>
hipError_t launch_logits_t(const G16Args& a, const HeadArgs& p, hipStream_t stream) {
  // raised once per process; the initialisation of a function-local static
  // is thread-safe, so concurrent first calls do not race
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&head_logits_kernel<T, kStore>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, kG16Lds);
  if (lds_limit != hipSuccess) return lds_limit;
  const Timer t(QK_HEAD_LOGITS, stream, true);
  const dim3 grid(static_cast<unsigned>((p.nv + kBN - 1) / kBN), static_cast<unsigned>((a.M + kBM - 1) / kBM));
  hipExtLaunchKernelGGL((head_logits_kernel<T, kStore>), grid, dim3(kThreads), kG16Lds, stream, t.start(), t.end(), 0, a, p);
  return hipGetLastError();
}

template <class T>
hipError_t launch_logits_split(const G16Args& a, const HeadArgs& p, hipStream_t stream) {
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&head_part_kernel<T>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, kG16Lds);
  if (lds_limit != hipSuccess) return lds_limit;
  const int64_t splits = (a.red + a.k_per - 1) / a.k_per;
  const dim3 grid(static_cast<unsigned>((p.nv + kBN - 1) / kBN), static_cast<unsigned>((a.M + kBM - 1) / kBM),
                  static_cast<unsigned>(splits));
  {
    const Timer t(QK_HEAD_LOGITS, stream, true);
    hipExtLaunchKernelGGL((head_part_kernel<T>), grid, dim3(kThreads), kG16Lds, stream, t.start(), t.end(), 0, a, p.ldp);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 units(static_cast<unsigned>((a.M * p.nh + 7) / 8));
  Timer tm(QK_REDUCE, stream);
  if (p.P != nullptr)
    hipLaunchKernelGGL((head_join_kernel<T, true>), units, dim3(256), 0, stream, a.part, splits, a.M, p);
  else
    hipLaunchKernelGGL((head_join_kernel<T, false>), units, dim3(256), 0, stream, a.part, splits, a.M, p);
  tm.stop();
  return hipGetLastError();
}

template <class T, bool kSplit>
hipError_t launch_dx_t(const G16Args& a, const DxArgs& p, hipStream_t stream) {
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&head_dx_kernel<T, kSplit>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, kG16Lds);
  if (lds_limit != hipSuccess) return lds_limit;
  const unsigned zs = static_cast<unsigned>(kSplit ? p.splits : 1);
  const dim3 grid(static_cast<unsigned>((p.K + kBN - 1) / kBN), static_cast<unsigned>((p.M + kBM - 1) / kBM), zs);
  const Timer t(QK_HEAD_DX, stream, true);
  hipExtLaunchKernelGGL((head_dx_kernel<T, kSplit>), grid, dim3(kThreads), kG16Lds, stream, t.start(), t.end(), 0, a, p);
  return hipGetLastError();
}
template <class T>
hipError_t launch_dx(const G16Args& a, const DxArgs& p, hipStream_t stream) {
  const hipError_t e = p.part != nullptr ? launch_dx_t<T, true>(a, p, stream) : launch_dx_t<T, false>(a, p, stream);
  if (e != hipSuccess || p.part == nullptr) return e;
  int64_t blocks = (p.M * p.K / 4 + 255) / 256;
  if (blocks > 8192) blocks = 8192;
  Timer tm(QK_REDUCE, stream);
  hipLaunchKernelGGL(head_sum_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p);
  tm.stop();
  return hipGetLastError();
}

template <class T>
hipError_t head_loss_t(int64_t M, int64_t K, int64_t V, const uint16_t* X, const uint16_t* W, const int64_t* targets,
                       const float* weights, int64_t ignore, float* loss, float* lse, uint16_t* dX, void* ws,
                       hipStream_t stream) {
  const HeadPlan h = head_plan(M, K, V, dX != nullptr);
  char* at = static_cast<char*>(ws);
  auto take = [&](int64_t bytes) {
    char* p = at;
    at += bytes;
    return p;
  };
  uint16_t* P = reinterpret_cast<uint16_t*>(take(h.p_bytes));
  float2* stats = reinterpret_cast<float2*>(take(h.stats_bytes));
  float2* run[2] = {reinterpret_cast<float2*>(take(h.row_bytes)), reinterpret_cast<float2*>(take(h.row_bytes))};
  float* st = reinterpret_cast<float*>(take(h.row_bytes));
  float* alpha = reinterpret_cast<float*>(take(h.row_bytes));
  float2* coef = reinterpret_cast<float2*>(take(h.row_bytes));
  float* lse_own = reinterpret_cast<float*>(take(h.row_bytes));
  float* sums = reinterpret_cast<float*>(take(h.sum_bytes));
  float* part = reinterpret_cast<float*>(take(h.part_bytes));
  for (int64_t i = 0; i < h.pieces; ++i) {
    const int64_t v0 = i * h.rows, nv = V - v0 < h.rows ? V - v0 : h.rows;
    const bool last = i + 1 == h.pieces;
    const bool logits_split = h.logits.splits > 1;
    const G16Args g{X, K, W + v0 * K, K, M, nv, K, nullptr, 0, nullptr, 0, logits_split ? part : nullptr, h.logits.k_per};
    HeadArgs p{targets, v0, nv, (nv + 63) / 64 * 64, V, ignore, dX != nullptr ? P : nullptr, stats, (nv + 127) / 128, st};
    hipError_t e = logits_split    ? launch_logits_split<T>(g, p, stream)
                   : dX != nullptr ? launch_logits_t<T, true>(g, p, stream)
                                   : launch_logits_t<T, false>(g, p, stream);
    if (e != hipSuccess) return e;
    RowArgs r{stats, p.nh, p.ldp, M, V, ignore, p.P, i > 0 ? run[(i + 1) & 1] : nullptr, run[i & 1], st, targets, weights,
              alpha, last ? loss : nullptr, lse != nullptr ? lse : lse_own, dX != nullptr ? coef : nullptr};
    // slices of a row until about 2048 workgroups, at least 2048 columns each
    int64_t slices = dX != nullptr ? (2048 + M - 1) / M : 1;
    if (slices > (p.ldp + 2047) / 2048) slices = (p.ldp + 2047) / 2048;
    {
      Timer tm(QK_HEAD_ROWS, stream);
      hipLaunchKernelGGL(head_rows_kernel<T>, dim3(static_cast<unsigned>(M), static_cast<unsigned>(slices)), dim3(256), 0,
                         stream, r);
      tm.stop();
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (dX == nullptr) continue;
    // the last piece may be shorter and need fewer splits
    const int64_t splits = (nv + h.k_per - 1) / h.k_per;
    const bool split = h.splits > 1;
    const G16Args w{P, p.ldp, W + v0 * K, K, M, K, nv, nullptr, 0, nullptr, 0, split ? part : nullptr, h.k_per};
    const DxArgs d{M, K, w.part, splits, i > 0 ? sums : nullptr, alpha, last ? nullptr : sums, coef, W, targets, dX,
                   1.0f / static_cast<float>(1 << head_shift<T>())};
    if ((e = launch_dx<T>(w, d, stream)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int64_t head_workspace_bytes(int64_t M, int64_t K, int64_t V, bool need_dx) { return head_plan(M, K, V, need_dx).total(); }

hipError_t launch_head_loss(int64_t M, int64_t K, int64_t V, const uint16_t* X, const uint16_t* W, const int64_t* targets,
                            const float* weights, int64_t ignore, float* loss, float* lse, uint16_t* dX, void* ws,
                            hipStream_t stream, int dtype) {
  return dtype == kDtypeF16 ? head_loss_t<F16>(M, K, V, X, W, targets, weights, ignore, loss, lse, dX, ws, stream)
                            : head_loss_t<Bf16>(M, K, V, X, W, targets, weights, ignore, loss, lse, dX, ws, stream);
}

}  // namespace qn
