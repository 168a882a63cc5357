// A step of the adapter along its orthogonalised momentum, for gfx950.  Per matrix
// (A: K x r, B: r x N), with g its gradient:
//   m <- mu m + (1 - mu) g,   u = (1 - mu) g + mu m  (Nesterov; else u = m),
//   X_0 = u / max(|u|, eps),  X <- a X + (b S + c S^2) X with S = X Xᵀ, `steps` times,
//   p <- p (1 - lr wd) - lr s X.
//
// The rank is small, so the iteration lives in r x r.  With U the matrix as long x r
// rows, every iterate is U times a polynomial of the Gram matrix G = Uᵀ U / |u|^2:
//   P = a I + b G + c G^2,   Q <- Q P,   G <- P G P,      X = U Q / |u|,
// and the long matrix is read twice (Gram, product) instead of twice a step.  G's
// rounding errors are absolute where the iteration on X itself has relative ones, and
// a small singular value's part of G grows by a^2 a step, twelvefold; G, Q and P are
// therefore 64-bit throughout (v_mfma_f64_16x16x4_f64), as are the sums of both long
// products.  A direction that U lacks has an eigenvalue of a few 2^-53 in G, of either
// sign; near -1, where no real one lies, the polynomial would run away (at the default
// coefficients after some 18 steps).  Steps end where a^(2 steps) passes 2^29: there the
// update is off by at most 1e-8 of its largest element, by 2e-12 after five default
// steps (U of rank 1 to 8, with equal columns, with singular values down to 1e-8).  The
// trace of U ᵀU is |u|^2, so the norm costs no pass of its own.
#include <cmath>

#include "common.hpp"
#include "kernels.hpp"
#include "side_jobs.hpp"

namespace qn {

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
int64_t align256(int64_t x) { return round_up(x, 256); }

typedef double f64x4 __attribute__((ext_vector_type(4)));

// One matrix of the step.  len: K or N; u: its update direction in the workspace, filled
// up with zeros: tall (A) len_p x rp, wide (B) rp x len_p.
struct MuonJob {
  uint16_t* param;
  const void* grad;
  float* mom;
  float* master;        // may be null
  float* u;
  double* part;         // Gram partials, by chunk
  double* mat;          // G, the next G, H, T, Q, the next Q: rp x rp each (r <= 64: G, Q alone)
  int64_t len, len_p;   // len_p: up to a multiple of 64
  int chunk, chunks;    // of len_p, elements a Gram workgroup takes
  int tall;
  double step;          // lr times the shape's factor
};
struct MuonArgs {
  MuonJob j[2];
  int r, rp, tiles;     // rp: r up to 16; tiles: 64-wide tiles of it
  int nesterov, steps;
  double momentum, decay, eps, a, b, c;   // decay: 1 - lr wd
};

__device__ __forceinline__ const MuonJob& job_of(const MuonArgs& p, int64_t first, int64_t& blk) {
  const bool second = blk >= first;
  if (second) blk -= first;
  return p.j[second];
}
__device__ __forceinline__ f64x4 mfma64(double a, double b, const f64x4& c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// The gradient's element type: NF4_AB_*.
template <int kGrad>
__device__ __forceinline__ float muon_grad(Rsrc r, uint32_t at) {
  if (kGrad == NF4_AB_F32) return ld_f32(r, at == kMasked ? kMasked : 4 * at);
  const uint32_t h = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, at == kMasked ? kMasked : 2 * at, 0, 0));
  return kGrad == NF4_AB_F16 ? F16::widen(h) : Bf16::widen(h);
}
// m updated and u, of an element.
struct MuonDirection {
  double mu, nu, ug, um;
  __device__ explicit MuonDirection(const MuonArgs& p)
      : mu(p.momentum), nu(1.0 - p.momentum), ug(p.nesterov ? nu : 0.0), um(p.nesterov ? mu : 1.0) {}
  __device__ __forceinline__ float step(float g, float& m) const {
    m = static_cast<float>(mu * m + nu * g);
    return static_cast<float>(ug * g + um * m);
  }
};

// Everybody's LDS accesses are done; stores to memory may be under way, which
// __syncthreads() would wait for.
__device__ __forceinline__ void meet_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// r <= 64.  Workgroup: one chunk of the long side; per 64 of it m and u, element by element
// in the order in memory, u into LDS as [long][rank], and its wave's 16 of the Gram
// matrix's upper tiles; the next 64 are requested meanwhile.  8192 and 22016 long at rank
// 64: 13 us for 15.5 MB read and 15.5 written (6 at a copy's rate), a workgroup a CU of two
// turns; with a branch around every element and nothing requested ahead 17.
template <int NT, int kGrad, bool kTall>
__device__ __forceinline__ void muon_gram64(const MuonArgs& p, const MuonJob& J, int64_t blk, float* tile, double* red) {
  constexpr int kPairs = NT * (NT + 1) / 2, kRp = 16 * NT, kLd = kRp + 1, kLoads = kRp / 4;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, q = lane & 15, g = lane >> 4;
  const int64_t beg = blk * J.chunk, end = min(J.len_p, beg + J.chunk), len_p = J.len_p;
  const uint32_t r = p.r, len = static_cast<uint32_t>(J.len);
  const Rsrc rg = make_rsrc(J.grad, int64_t(r) * len * (kGrad == NF4_AB_F32 ? 4 : 2)), rm = make_rsrc(J.mom, int64_t(r) * len * 4);
  const MuonDirection dir(p);
  float* const u_out = J.u;
  auto place = [&](int k, int& l, int& c) {   // this thread's k-th element: long l0 + l, rank c
    const int e = t + 256 * k;
    l = kTall ? e / kRp : e & 63;
    c = kTall ? e - l * kRp : e >> 6;
  };
  struct Loads {
    float g[kLoads], m[kLoads];
    uint32_t at[kLoads];
  };
  auto load = [&](int64_t l0, Loads& v) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      int l, c;
      place(k, l, c);
      const uint32_t L = static_cast<uint32_t>(l0) + l;
      v.at[k] = L < len && c < static_cast<int>(r) ? (kTall ? L * r + c : c * len + L) : kMasked;
      v.g[k] = muon_grad<kGrad>(rg, v.at[k]);
      v.m[k] = ld_f32(rm, v.at[k] == kMasked ? kMasked : 4 * v.at[k]);
    }
  };
  f64x4 acc[kPairs];
#pragma unroll
  for (int x = 0; x < kPairs; ++x) acc[x] = f64x4{0, 0, 0, 0};
  Loads v;
  load(beg, v);
  for (int64_t l0 = beg; l0 < end; l0 += 64) {
    meet_lds();   // the last 64 have been multiplied
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      int l, c;
      place(k, l, c);
      // masked elements are zeros, whose u is zero, and a masked store is dropped
      const float u = dir.step(v.g[k], v.m[k]);
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v.m[k]), rm, v.at[k] == kMasked ? kMasked : 4 * v.at[k], 0, 0);
      u_out[kTall ? (l0 + l) * kRp + c : c * len_p + l0 + l] = u;
      tile[l * kLd + c] = u;
    }
    if (l0 + 64 < end) load(l0 + 64, v);
    meet_lds();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      double f[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) f[i] = static_cast<double>(tile[(16 * wave + 4 * s + g) * kLd + 16 * i + q]);
#pragma unroll
      for (int i = 0, x = 0; i < NT; ++i)
#pragma unroll
        for (int j = i; j < NT; ++j, ++x) acc[x] = mfma64(f[i], f[j], acc[x]);
    }
  }
  // lane: rows 16 i + g + 4 e, column 16 j + q
  // the sum of the waves, (0 + 2) + (1 + 3)
#pragma unroll
  for (int w = 0; w < 4; w += 2) {
    if ((wave & 2) == w) {
#pragma unroll
      for (int x = 0; x < kPairs; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          double& at = red[((wave & 1) * kPairs + x) * 256 + (g + 4 * e) * 16 + q];
          at = w == 0 ? acc[x][e] : at + acc[x][e];
        }
    }
    meet_lds();
  }
  double* part = J.part + blk * (kPairs * 256);
  for (int i = t; i < kPairs * 256; i += 256) part[i] = red[i] + red[kPairs * 256 + i];
}
template <int NT, int kGrad>
__global__ __launch_bounds__(256) void muon_gram64_kernel(MuonArgs p, int64_t first) {
  constexpr int kPairs = NT * (NT + 1) / 2;
  __shared__ float tile[64 * (16 * NT + 1)];
  __shared__ double red[2 * kPairs * 256];
  const int64_t blk = blockIdx.x;
  if (blk < first) muon_gram64<NT, kGrad, true>(p, p.j[0], blk, tile, red);
  else muon_gram64<NT, kGrad, false>(p, p.j[1], blk - first, tile, red);
}

// r > 64: m and u, element by element of the filled-up matrix; 11 us at 8192 and 22016 long,
// rank 128 (62 MB), 20 at 256: a copy's rate or a little more.
template <int kGrad>
__global__ __launch_bounds__(256) void muon_momentum_kernel(MuonArgs p, int64_t first) {
  int64_t blk = blockIdx.x;
  const MuonJob& J = job_of(p, first, blk);
  const MuonDirection dir(p);
  float* const u_out = J.u;
  const uint32_t row_p = J.tall ? p.rp : static_cast<uint32_t>(J.len_p);
  const uint32_t rows = J.tall ? static_cast<uint32_t>(J.len) : p.r, cols = J.tall ? p.r : static_cast<uint32_t>(J.len);
  const uint32_t count = static_cast<uint32_t>(J.len_p * p.rp);
  const Rsrc rg = make_rsrc(J.grad, int64_t(rows) * cols * (kGrad == NF4_AB_F32 ? 4 : 2)), rm = make_rsrc(J.mom, int64_t(rows) * cols * 4);
  float g[4], m[4];
  uint32_t at[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t i = static_cast<uint32_t>(blk) * 1024 + k * 256 + threadIdx.x, y = i / row_p, x = i - y * row_p;
    at[k] = i < count && y < rows && x < cols ? y * cols + x : kMasked;
    g[k] = muon_grad<kGrad>(rg, at[k]);
    m[k] = ld_f32(rm, at[k] == kMasked ? kMasked : 4 * at[k]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t i = static_cast<uint32_t>(blk) * 1024 + k * 256 + threadIdx.x;
    const float u = dir.step(g[k], m[k]);   // zero where masked
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, m[k]), rm, at[k] == kMasked ? kMasked : 4 * at[k], 0, 0);
    if (i < count) u_out[i] = u;
  }
}

// Four Gram operands of a 16-deep step: element (l0 + .., 16 i + q) of U; which four of
// the sixteen a lane holds in step s does not matter as long as both operands agree.
__device__ __forceinline__ void gram_load(const MuonJob& J, int rp, int64_t l0, int col, int q, int g, float (&v)[4]) {
  if (col + q >= rp) {   // tiles of 64 past the filled-up rank
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = 0.0f;
  } else if (J.tall) {
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = J.u[(l0 + 4 * s + g) * rp + col + q];
  } else {
    const float4 f = *reinterpret_cast<const float4*>(J.u + (col + q) * J.len_p + l0 + 4 * g);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  }
}

// r > 64.  Workgroup: one 64 x 64 tile pair (I <= J) of the Gram matrix over one chunk; its
// waves take every fourth 16 and are added in LDS in order.  8192 and 22016 long: 29 us at
// rank 128, 77 at 256, the 64-bit matrix unit busy for 36 and 44 % of it; each pair reads its
// rows of U again (31 and 124 MB, most of it from the caches).
__global__ __launch_bounds__(256) void muon_gram_kernel(MuonArgs p, int64_t first) {
  __shared__ double red[64 * 64];
  int64_t blk = blockIdx.x;
  const MuonJob& J = job_of(p, first, blk);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, q = lane & 15, g = lane >> 4;
  const int pairs = p.tiles * (p.tiles + 1) / 2;
  const int64_t chunk = blk / pairs;
  int pair = static_cast<int>(blk - chunk * pairs), I = 0;
  while (pair >= p.tiles - I) pair -= p.tiles - I++;
  const int ci = 64 * I, cj = 64 * (I + pair);
  f64x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f64x4{0, 0, 0, 0};
  const int64_t end = min(J.len_p, (chunk + 1) * J.chunk);
  for (int64_t l0 = chunk * J.chunk + 16 * wave; l0 < end; l0 += 64) {
    float a[4][4], b[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      gram_load(J, p.rp, l0, ci + 16 * i, q, g, a[i]);
      gram_load(J, p.rp, l0, cj + 16 * i, q, g, b[i]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma64(static_cast<double>(a[i][s]), static_cast<double>(b[j][s]), acc[i][j]);
  }
  // lane: rows 16 i + g + 4 e, column 16 j + q
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            double& at = red[(16 * i + g + 4 * e) * 64 + 16 * j + q];
            at = w == 0 ? acc[i][j][e] : at + acc[i][j][e];
          }
    }
    __syncthreads();
  }
  double* out = J.part + blk * 4096;
  for (int i = t; i < 4096; i += 256) out[i] = red[i];
}

// G (both halves) from the partials: a workgroup adds 32 elements, each of its eight rows of
// threads the chunks x, x + 8, .., and then the eight in order.  kSide: tiles of 16 (r <= 64,
// with `side` of them) or of 64.
template <int kSide>
__global__ __launch_bounds__(256) void muon_sum_kernel(MuonArgs p, int side, int64_t first) {
  __shared__ double red[8][32];
  int64_t blk = blockIdx.x;
  const MuonJob& J = job_of(p, first, blk);
  const int pairs = side * (side + 1) / 2, plane = pairs * kSide * kSide;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, at = static_cast<int>(blk) * 32 + x;
  double s = 0.0;
#pragma unroll 4
  for (int c = y; c < J.chunks; c += 8) s += J.part[static_cast<int64_t>(c) * plane + at];
  red[y][x] = s;
  __syncthreads();
  if (y != 0) return;
  for (int k = 1; k < 8; ++k) s += red[k][x];
  int pair = at / (kSide * kSide), I = 0;
  while (pair >= side - I) pair -= side - I++;
  const int i = kSide * I + (at / kSide) % kSide, j = kSide * (I + pair) + at % kSide;
  if (i >= p.rp || j >= p.rp) return;
  J.mat[i * p.rp + j] = s;
  J.mat[j * p.rp + i] = s;
}

// 1 / max(|u|, eps)^2 from the Gram matrix's diagonal (d: its first element, rows ld apart);
// NaN where u is not finite, which 1 / infinity would hide from an update without a step.
__device__ __forceinline__ double muon_scale(const double* d, int ld, int rp, double eps) {
  double s = 0.0;
  for (int i = threadIdx.x & 63; i < rp; i += 64) s += d[i * (ld + 1)];
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) s += __shfl_xor(s, x, 64);
  const double n = sqrt(s), m = n > eps ? n : (n == n ? eps : n);
  return (1.0 + 0.0 * n) / (m * m);
}

// r <= 64: the whole iteration of one matrix in one workgroup, G, P, Q and S = G P in LDS.
// Everything is symmetric, so only the upper tiles are computed, a wave each, and stored
// twice; all operands are read along their rows (68 a row: 64 lanes on all banks), P's
// once for its three products.  Bound by the matrix unit of one CU, 32 flops a cycle and
// SIMD: at r = 64 the 17 products, 64 deep, three tiles a SIMD, take 22 us of the 41; LDS
// reads take about 7, the rest are 15 barriers, start and end.  More CUs would meet in
// memory three times a step, at 2 to 3 us each.
template <int NT>
__global__ __launch_bounds__(64 * (NT * (NT + 1) / 2)) void muon_iterate64_kernel(MuonArgs p) {
  constexpr int kRp = 16 * NT, kLd = 68, kThreads = 64 * (NT * (NT + 1) / 2), kDeep = kRp / 4;
  extern __shared__ double lds[];
  double *G = lds, *P = G + kRp * kLd, *Q = P + kRp * kLd, *S = Q + kRp * kLd;
  double* mat = p.j[blockIdx.x].mat;
  const int t = threadIdx.x, lane = t & 63, q = lane & 15, g = lane >> 4;
  int pair = __builtin_amdgcn_readfirstlane(t >> 6), I = 0;
  while (pair >= NT - I) pair -= NT - I++;
  const int i0 = 16 * I, j0 = 16 * (I + pair);
  for (int i = t; i < kRp * kRp; i += kThreads) G[(i / kRp) * kLd + i % kRp] = mat[i];
  __syncthreads();
  const double sc = muon_scale(G, kLd, kRp, p.eps);
  __syncthreads();
  for (int i = t; i < kRp * kRp; i += kThreads) {
    const int at = (i / kRp) * kLd + i % kRp;
    G[at] *= sc;
    Q[at] = i / kRp == i % kRp ? 1.0 : 0.0;
  }
  __syncthreads();
  const int ra = (i0 + q) * kLd + g, rb = (j0 + q) * kLd + g;
  auto put = [&](double* M, const f64x4& v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + g + 4 * e, j = j0 + q;
      if (i > j) continue;   // a diagonal tile's lower half comes from its upper
      M[i * kLd + j] = v[e];
      M[j * kLd + i] = v[e];
    }
  };
  struct Rows {
    double v[kDeep];
  };
  auto rows = [&](const double* at) {
    Rows R;
#pragma unroll
    for (int k = 0; k < kDeep; ++k) R.v[k] = at[4 * k];
    return R;
  };
  // two chains, so that a wave need not wait for its own last product
  auto product = [&](const Rows& a, const Rows& b) {
    f64x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kDeep; k += 2) {
      x = mfma64(a.v[k], b.v[k], x);
      y = mfma64(a.v[k + 1], b.v[k + 1], y);
    }
    return x + y;
  };
  f64x4 gt;   // this wave's tile of G
#pragma unroll
  for (int e = 0; e < 4; ++e) gt[e] = G[(i0 + g + 4 * e) * kLd + j0 + q];
  for (int step = 0; step < p.steps; ++step) {
    const bool last = step + 1 == p.steps;
    const Rows ga = rows(G + ra);
    f64x4 pt = product(ga, rows(G + rb));
#pragma unroll
    for (int e = 0; e < 4; ++e) pt[e] = (i0 + g + 4 * e == j0 + q ? p.a : 0.0) + p.b * gt[e] + p.c * pt[e];
    put(P, pt);
    __syncthreads();
    const Rows pb = rows(P + rb);
    f64x4 qt = pt;
    if (step > 0) qt = product(rows(Q + ra), pb);
    if (!last) put(S, product(ga, pb));
    __syncthreads();
    put(Q, qt);          // read again after the next barrier but one
    if (last) break;
    gt = product(rows(S + ra), pb);
    put(G, gt);          // read before the last barrier
    __syncthreads();
  }
  __syncthreads();
  // Q / |u|, after G
  const double root = sqrt(sc);
  for (int i = t; i < kRp * kRp; i += kThreads) mat[kRp * kRp + i] = root * Q[(i / kRp) * kLd + i % kRp];
}

// r > 64: which r x r products a launch computes: H = G G; T = G P and the next Q = Q P; the
// next G = T P.
enum { kSquare = 0, kMixed = 1, kNext = 2 };

// Workgroup: one upper 16 x 16 tile, stored twice (everything is symmetric; both operands are
// read along their rows); its waves every fourth 16 of the depth, all rows requested at
// once, since what the launch before wrote comes from far, and added in LDS in order.
// (A wave a tile, 16 requests after another: 10 to 19 us a launch at r = 256, now 7 to 12.)
// kFirst: G carries its scale still, Q is the identity.  The last step's Q gets its 1 / |u|.
template <int kWhat, bool kFirst>
__global__ __launch_bounds__(256) void muon_product_kernel(MuonArgs p, int step, const double* scales, int64_t first) {
  constexpr bool kQ = kWhat == kMixed && !kFirst;
  __shared__ f64x4 red[kQ ? 2 : 1][4][64];
  int64_t blk = blockIdx.x;
  const bool second = blk >= first;
  const MuonJob& J = job_of(p, first, blk);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane & 15, g = lane >> 4, rp = p.rp, side = rp / 16;
  const int plane = rp * rp;
  const int now = step & 1, then = 1 - now;
  const double *G = J.mat + now * plane, *Q = J.mat + (4 + now) * plane;
  double *H = J.mat + 2 * plane, *T = J.mat + 3 * plane, *Gn = J.mat + then * plane, *Qn = J.mat + (4 + then) * plane;
  const double sc = scales[second], g1 = kFirst ? sc : 1.0;
  int pair = static_cast<int>(blk), I = 0;
  while (pair >= side - I) pair -= side - I++;
  const int i0 = 16 * I, j0 = 16 * (I + pair);
  struct Rows {
    f64x4 a, b, h, q;
  };
  Rows R[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = 16 * (4 * u + wave) + 4 * g, ia = (i0 + q) * rp + k, jb = (j0 + q) * rp + k;
    if (16 * (4 * u + wave) >= rp) break;
    R[u].a = *reinterpret_cast<const f64x4*>((kWhat == kNext ? T : G) + ia);
    R[u].b = *reinterpret_cast<const f64x4*>(G + jb);
    if (kWhat != kSquare) R[u].h = *reinterpret_cast<const f64x4*>(H + jb);
    if (kQ) R[u].q = *reinterpret_cast<const f64x4*>(Q + ia);
  }
  f64x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (16 * (4 * u + wave) >= rp) break;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const double gi = kWhat == kNext ? R[u].a[s] : g1 * R[u].a[s];
      const double oj = kWhat == kSquare
                            ? g1 * R[u].b[s]
                            : (16 * (4 * u + wave) + 4 * g + s == j0 + q ? p.a : 0.0) + p.b * g1 * R[u].b[s] + p.c * R[u].h[s];
      x = mfma64(gi, oj, x);
      if (kQ) y = mfma64(R[u].q[s], oj, y);
    }
  }
  red[0][wave][lane] = x;
  if (kQ) red[kQ][wave][lane] = y;
  __syncthreads();
  if (wave != 0) return;
  for (int w = 1; w < 4; ++w) {
    x += red[0][w][lane];
    if (kQ) y += red[kQ][w][lane];
  }
  double* out = kWhat == kSquare ? H : (kWhat == kMixed ? T : Gn);
  const double root = step + 1 == p.steps ? sqrt(sc) : 1.0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = i0 + g + 4 * e, j = j0 + q;
    if (i > j) continue;
    if (kWhat == kMixed) {
      const double v = root * (kFirst ? (i == j ? p.a : 0.0) + p.b * g1 * G[i * rp + j] + p.c * H[i * rp + j] : y[e]);
      Qn[i * rp + j] = v;
      Qn[j * rp + i] = v;
    }
    out[i * rp + j] = x[e];
    out[j * rp + i] = x[e];
  }
}

// r > 64: the scales of both matrices; without a step also Q.
__global__ __launch_bounds__(64) void muon_scale_kernel(MuonArgs p, double* scales) {
  const int rp = p.rp;
  const double s = muon_scale(p.j[blockIdx.x].mat, rp, rp, p.eps);
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
  if (p.steps == 0)
    for (int i = threadIdx.x; i < rp * rp; i += 64) p.j[blockIdx.x].mat[4 * rp * rp + i] = i / rp == i % rp ? sqrt(s) : 0.0;
}

// X = U Q and the parameters.  Workgroup: 64 of the long side, a wave 16; Q (symmetric, so
// both layouts read it along its rows) passes through LDS in 64 x 64 pieces.  Bound by
// memory: u, the parameters and their copies once (27 MB at 8192 and 22016 long, rank 64:
// 15.5 us, of it two waits for memory and 3.4 us of 64-bit products).  Above rank 64 by its
// products and what feeds them, 44 us at rank 128 and 150 at 256: the matrix unit busy for 34
// and 38 % of it, the vector units (u to 64 bits, addresses) for half, u read once per 64 of
// the rank.
template <bool kF16, bool kMaster, bool kTall>
__device__ __forceinline__ void muon_apply(const MuonArgs& p, const MuonJob& J, int64_t blk, const double* Q, double* qs) {
  constexpr int kLd = 65;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, q = lane & 15, g = lane >> 4, rp = p.rp;
  const int64_t l0 = blk * 64 + 16 * wave;
  const uint32_t r = p.r, len = static_cast<uint32_t>(J.len);
  const Rsrc rq = make_rsrc(Q, static_cast<int64_t>(rp) * rp * 8);
  const Rsrc ro = make_rsrc(kMaster ? static_cast<const void*>(J.master) : J.param, int64_t(r) * len * (kMaster ? 4 : 2));
  for (int c0 = 0; c0 < rp; c0 += 64) {
    const int cn = min(rp - c0, 64);
    // the old values of this lane's outputs.  tall: long g + 4 e, rank q; wide: the other way
    uint32_t at[4][4];
    float old[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t l = static_cast<uint32_t>(l0) + (kTall ? g + 4 * e : q), c = c0 + 16 * j + (kTall ? q : g + 4 * e);
        at[j][e] = l < len && c < r ? (kTall ? l * r + c : c * len + l) : kMasked;
        old[j][e] = muon_grad<kMaster ? NF4_AB_F32 : (kF16 ? NF4_AB_F16 : NF4_AB_BF16)>(ro, at[j][e]);
      }
    f64x4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = f64x4{0, 0, 0, 0};
    for (int k0 = 0; k0 < rp; k0 += 64) {
      const int kn = min(rp - k0, 64);
      float u[4][4];
      // u, filled up, may pass 2 GiB; past kn the last 16 again, unused
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int64_t k = k0 + min(16 * kk, kn - 16);
        if constexpr (kTall) {
          const float4 v = *reinterpret_cast<const float4*>(J.u + (l0 + q) * rp + k + 4 * g);
          u[kk][0] = v.x;
          u[kk][1] = v.y;
          u[kk][2] = v.z;
          u[kk][3] = v.w;
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s) u[kk][s] = J.u[(k + 4 * s + g) * J.len_p + l0 + q];
        }
      }
      uint2 qv[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int c = (t >> 6) + 4 * i, k = t & 63;
        qv[i] = ld_b64(rq, c < cn && k < kn ? static_cast<uint32_t>((c0 + c) * rp + k0 + k) * 8 : kMasked);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 16; ++i) qs[((t >> 6) + 4 * i) * kLd + (t & 63)] = __builtin_bit_cast(double, qv[i]);
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (16 * kk >= kn) break;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = 16 * kk + (kTall ? 4 * g + s : 4 * s + g);
          const double ud = static_cast<double>(u[kk][s]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (16 * j >= cn) break;
            const double w = qs[(16 * j + q) * kLd + k];
            x[j] = kTall ? mfma64(ud, w, x[j]) : mfma64(w, ud, x[j]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (at[j][e] == kMasked) continue;
        const float v = static_cast<float>(static_cast<double>(old[j][e]) * p.decay - J.step * x[j][e]);
        if (kMaster) J.master[at[j][e]] = v;
        J.param[at[j][e]] = half_of(v, kF16);
      }
  }
}
template <bool kF16, bool kMaster>
__global__ __launch_bounds__(256) void muon_apply_kernel(MuonArgs p, int q_at, int64_t first) {
  __shared__ double qs[64 * 65];
  const int64_t blk = blockIdx.x, q0 = static_cast<int64_t>(q_at) * p.rp * p.rp;
  if (blk < first) muon_apply<kF16, kMaster, true>(p, p.j[0], blk, p.j[0].mat + q0, qs);
  else muon_apply<kF16, kMaster, false>(p, p.j[1], blk - first, p.j[1].mat + q0, qs);
}

struct MuonSizes {
  int64_t len_p, u, part, mat;
  int chunk, chunks;
};
// Chunks of both matrices so that about 256 workgroups run.
MuonSizes muon_sizes(int64_t len, int64_t other, int64_t r) {
  MuonSizes s;
  const int64_t rp = round_up(r, 16), tiles = cdiv(rp, 64), pairs = tiles * (tiles + 1) / 2;
  s.len_p = round_up(len, 64);
  const int64_t chunk = round_up(cdiv(s.len_p + round_up(other, 64), cdiv(256, pairs)), 64);
  s.chunk = static_cast<int>(chunk);
  s.chunks = static_cast<int>(cdiv(s.len_p, chunk));
  const int64_t side = rp / 16;
  const int64_t plane = tiles == 1 ? side * (side + 1) / 2 * 256 : pairs * 4096;
  s.u = align256(s.len_p * rp * 4);
  s.part = align256(s.chunks * plane * 8);
  s.mat = align256((tiles == 1 ? 2 : 6) * rp * rp * 8);
  return s;
}

template <int NT>
hipError_t launch_muon64(const MuonArgs& p, int grad, int64_t c0, int64_t c1, hipStream_t stream) {
  constexpr int kPairs = NT * (NT + 1) / 2, kLds = 4 * 16 * NT * 68 * 8;
  static const hipError_t lds_limit = hipFuncSetAttribute(reinterpret_cast<const void*>(&muon_iterate64_kernel<NT>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (lds_limit != hipSuccess) return lds_limit;
  auto* k = grad == NF4_AB_F32 ? muon_gram64_kernel<NT, NF4_AB_F32>
                               : (grad == NF4_AB_F16 ? muon_gram64_kernel<NT, NF4_AB_F16> : muon_gram64_kernel<NT, NF4_AB_BF16>);
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(c0 + c1)), dim3(256), 0, stream, p, c0);
  hipLaunchKernelGGL(muon_sum_kernel<16>, dim3(2 * kPairs * 8), dim3(256), 0, stream, p, NT, int64_t(kPairs) * 8);
  hipLaunchKernelGGL(muon_iterate64_kernel<NT>, dim3(2), dim3(64 * kPairs), kLds, stream, p);
  return hipGetLastError();
}

}  // namespace

int64_t muon_workspace_bytes(int64_t K, int64_t N, int64_t r) {
  const MuonSizes a = muon_sizes(K, N, r), b = muon_sizes(N, K, r);
  return 256 + a.u + a.part + a.mat + b.u + b.part + b.mat;
}

hipError_t launch_muon(int64_t K, int64_t N, int64_t r, uint16_t* A, uint16_t* B, const void* dA, const void* dB,
                       float* mA, float* mB, float* A_master, float* B_master, const qlora_muon_t& o, void* ws,
                       hipStream_t stream, int dtype, bool grad16) {
  MuonArgs p{};
  p.r = static_cast<int>(r);
  p.rp = static_cast<int>(round_up(r, 16));
  p.tiles = (p.rp + 63) / 64;
  const bool f16 = dtype == kDtypeF16;
  const int grad = !grad16 ? NF4_AB_F32 : (f16 ? NF4_AB_F16 : NF4_AB_BF16);
  p.momentum = o.momentum;
  p.decay = 1.0 - o.lr * o.weight_decay;
  p.nesterov = o.nesterov != 0;
  p.steps = o.steps;
  // a norm is zero or at least an fp32 number's 2^-149; kept where 1 / eps^2 is finite too
  p.eps = std::fmax(o.eps, 1e-60);
  p.a = o.a;
  p.b = o.b;
  p.c = o.c;
  double* scales = static_cast<double*>(ws);
  char* at = static_cast<char*>(ws) + 256;
  MuonSizes s[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t len = i ? N : K;
    s[i] = muon_sizes(len, i ? K : N, r);
    MuonJob& J = p.j[i];
    J.param = i ? B : A;
    J.grad = i ? dB : dA;
    J.mom = i ? mB : mA;
    J.master = i ? B_master : A_master;
    J.len = len;
    J.len_p = s[i].len_p;
    J.chunk = s[i].chunk;
    J.chunks = s[i].chunks;
    J.tall = i == 0;
    const double rows = i ? r : K, cols = i ? N : r;
    const double f = o.scaling == NF4_MUON_SCALE_SPECTRAL ? std::sqrt(std::fmax(1.0, rows / cols))
                     : o.scaling == NF4_MUON_SCALE_RMS    ? 0.2 * std::sqrt(std::fmax(rows, cols))
                                                          : 1.0;
    J.step = o.lr * f;
    J.u = reinterpret_cast<float*>(at);
    at += s[i].u;
    J.part = reinterpret_cast<double*>(at);
    at += s[i].part;
    J.mat = reinterpret_cast<double*>(at);
    at += s[i].mat;
  }
  auto grid = [](int64_t a, int64_t b) { return dim3(static_cast<unsigned>(a + b)); };
  Timer tm(QK_MUON, stream);
  int q_at = 1;
  if (p.tiles == 1) {
    hipError_t e;
    switch (p.rp / 16) {
      case 1: e = launch_muon64<1>(p, grad, s[0].chunks, s[1].chunks, stream); break;
      case 2: e = launch_muon64<2>(p, grad, s[0].chunks, s[1].chunks, stream); break;
      case 3: e = launch_muon64<3>(p, grad, s[0].chunks, s[1].chunks, stream); break;
      default: e = launch_muon64<4>(p, grad, s[0].chunks, s[1].chunks, stream); break;
    }
    if (e != hipSuccess) return e;
  } else {
    const int64_t pairs = static_cast<int64_t>(p.tiles) * (p.tiles + 1) / 2;
    const int64_t m0 = cdiv(s[0].len_p * p.rp, 1024), m1 = cdiv(s[1].len_p * p.rp, 1024);
    auto* mk = grad == NF4_AB_F32 ? muon_momentum_kernel<NF4_AB_F32>
                                  : (grad == NF4_AB_F16 ? muon_momentum_kernel<NF4_AB_F16> : muon_momentum_kernel<NF4_AB_BF16>);
    hipLaunchKernelGGL(mk, grid(m0, m1), dim3(256), 0, stream, p, m0);
    hipLaunchKernelGGL(muon_gram_kernel, grid(s[0].chunks * pairs, s[1].chunks * pairs), dim3(256), 0, stream, p, s[0].chunks * pairs);
    hipLaunchKernelGGL(muon_sum_kernel<64>, grid(pairs * 128, pairs * 128), dim3(256), 0, stream, p, p.tiles, pairs * 128);
    hipLaunchKernelGGL(muon_scale_kernel, dim3(2), dim3(64), 0, stream, p, scales);
    const int64_t side = p.rp / 16, wgs = side * (side + 1) / 2;
    auto product = [&](auto* k, int i) {
      hipLaunchKernelGGL(k, grid(wgs, wgs), dim3(256), 0, stream, p, i, static_cast<const double*>(scales), wgs);
    };
    for (int i = 0; i < o.steps; ++i) {
      product(i == 0 ? muon_product_kernel<kSquare, true> : muon_product_kernel<kSquare, false>, i);
      product(i == 0 ? muon_product_kernel<kMixed, true> : muon_product_kernel<kMixed, false>, i);
      if (i + 1 < o.steps) product(i == 0 ? muon_product_kernel<kNext, true> : muon_product_kernel<kNext, false>, i);
    }
    q_at = 4 + (o.steps & 1);
  }
  auto* ak = f16 ? (A_master ? muon_apply_kernel<true, true> : muon_apply_kernel<true, false>)
                 : (A_master ? muon_apply_kernel<false, true> : muon_apply_kernel<false, false>);
  hipLaunchKernelGGL(ak, grid(s[0].len_p / 64, s[1].len_p / 64), dim3(256), 0, stream, p, q_at, s[0].len_p / 64);
  tm.stop();
  return hipGetLastError();
}

}  // namespace qn
