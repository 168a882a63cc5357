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
// a small singular value's part of G grows twelvefold a step; G, Q and P are
// therefore 64-bit throughout (v_mfma_f64_16x16x4_f64; an error of 2^-53 comes out below
// 1e-10), as are the sums of both long products.  The trace of U ᵀU is |u|^2, so the
// norm costs no pass of its own.
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
  double* part;         // Gram partials [chunks][pairs][64][64]
  double* mat;          // G, the next G, H, T, Q, the next Q: rp x rp each
  int64_t len, len_p;
  int64_t chunk;        // of len_p, elements a Gram workgroup takes
  int chunks, tall;
  double step;          // lr times the shape's factor
};
struct MuonArgs {
  MuonJob j[2];
  int r, rp, tiles;     // rp: r up to 16; tiles: 64-wide tiles of it
  int f16, grad16;
  int nesterov;
  double momentum, decay, eps, a, b, c;   // decay: 1 - lr wd
};

__device__ __forceinline__ const MuonJob& job_of(const MuonArgs& p, int64_t first, int64_t& blk) {
  const bool second = blk >= first;
  if (second) blk -= first;
  return p.j[second];
}

// m and u, element by element of the filled-up matrix.
__global__ __launch_bounds__(256) void muon_momentum_kernel(MuonArgs p, int64_t first) {
  int64_t blk = blockIdx.x;
  const MuonJob& J = job_of(p, first, blk);
  const uint32_t row_p = J.tall ? p.rp : static_cast<uint32_t>(J.len_p);
  const uint32_t rows = J.tall ? static_cast<uint32_t>(J.len) : p.r, cols = J.tall ? p.r : static_cast<uint32_t>(J.len);
  const int64_t count = J.len_p * p.rp;
  const double mu = p.momentum, nu = 1.0 - mu;
  for (int k = 0; k < 4; ++k) {
    const int64_t i = blk * 1024 + k * 256 + threadIdx.x;
    if (i >= count) return;
    const uint32_t y = static_cast<uint32_t>(i) / row_p, x = static_cast<uint32_t>(i) - y * row_p;
    float u = 0.0f;
    if (y < rows && x < cols) {
      const int64_t at = static_cast<int64_t>(y) * cols + x;
      const float g = p.grad16 ? widen_of(static_cast<const uint16_t*>(J.grad)[at], p.f16) : static_cast<const float*>(J.grad)[at];
      const float m = static_cast<float>(mu * J.mom[at] + nu * g);
      J.mom[at] = m;
      u = p.nesterov ? static_cast<float>(nu * g + mu * m) : m;
    }
    J.u[i] = u;
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

// Workgroup: one 64 x 64 tile pair (I <= J) of the Gram matrix over one chunk; its waves
// take every fourth 16 and are added in LDS in order.
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
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(static_cast<double>(a[i][s]), static_cast<double>(b[j][s]), acc[i][j], 0, 0, 0);
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

// G (both halves) from the partials, in order of the chunks.
__global__ __launch_bounds__(256) void muon_sum_kernel(MuonArgs p, int64_t first) {
  int64_t blk = blockIdx.x;
  const MuonJob& J = job_of(p, first, blk);
  const int pairs = p.tiles * (p.tiles + 1) / 2;
  const int at = static_cast<int>(blk) * 256 + threadIdx.x;   // of pairs * 4096
  double s = 0.0;
  for (int c = 0; c < J.chunks; ++c) s += J.part[static_cast<int64_t>(c) * pairs * 4096 + at];
  int pair = at >> 12, I = 0;
  while (pair >= p.tiles - I) pair -= p.tiles - I++;
  const int i = 64 * I + ((at >> 6) & 63), j = 64 * (I + pair) + (at & 63);
  if (i >= p.rp || j >= p.rp) return;
  J.mat[i * p.rp + j] = s;
  J.mat[j * p.rp + i] = s;
}

// 1 / max(|u|, eps)^2 from the Gram matrix's diagonal.
__device__ __forceinline__ double muon_scale(const double* G, int rp, double eps) {
  double s = 0.0;
  for (int i = threadIdx.x & 63; i < rp; i += 64) s += G[i * rp + i];
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) s += __shfl_xor(s, x, 64);
  const double n = sqrt(s), m = n > eps ? n : (n == n ? eps : n);
  return 1.0 / (m * m);
}

// Which r x r products a launch computes: H = G G; T = G P and the next Q = Q P; the
// next G = T P.
enum { kSquare = 0, kMixed = 1, kNext = 2 };

// A wave: one 16 x 16 tile.  All operands are symmetric up to rounding, so both are read
// along their rows.  step 0: G carries its scale still, Q is the identity.
__global__ __launch_bounds__(256) void muon_product_kernel(MuonArgs p, int what, int step, int64_t first) {
  int64_t blk = blockIdx.x;
  const MuonJob& J = job_of(p, first, blk);
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4, rp = p.rp, side = rp / 16;
  const int plane = rp * rp;
  const int now = step & 1, then = 1 - now;
  const double *G = J.mat + now * plane, *Q = J.mat + (4 + now) * plane;
  double *H = J.mat + 2 * plane, *T = J.mat + 3 * plane, *Gn = J.mat + then * plane, *Qn = J.mat + (4 + then) * plane;
  const double sc = step == 0 ? muon_scale(G, rp, p.eps) : 1.0;
  const int tile = static_cast<int>(blk) * 4 + (threadIdx.x >> 6);
  if (tile >= side * side) return;
  const int i0 = 16 * (tile / side), j0 = 16 * (tile % side);
  auto poly = [&](int i, int j) { return (i == j ? p.a : 0.0) + p.b * sc * G[i * rp + j] + p.c * H[i * rp + j]; };
  f64x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
  for (int k0 = 0; k0 < rp; k0 += 16) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + 4 * g + s;
      const double gi = what == kNext ? T[(i0 + q) * rp + k] : sc * G[(i0 + q) * rp + k];
      const double oj = what == kSquare ? sc * G[(j0 + q) * rp + k] : poly(j0 + q, k);
      x = __builtin_amdgcn_mfma_f64_16x16x4f64(gi, oj, x, 0, 0, 0);
      if (what == kMixed && step > 0) y = __builtin_amdgcn_mfma_f64_16x16x4f64(Q[(i0 + q) * rp + k], oj, y, 0, 0, 0);
    }
  }
  double* out = what == kSquare ? H : (what == kMixed ? T : Gn);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = i0 + g + 4 * e, j = j0 + q;
    if (what == kMixed) Qn[i * rp + j] = step == 0 ? poly(i, j) : y[e];
    out[i * rp + j] = x[e];
  }
}

// X = U Q / |u| and the parameters.
__device__ __forceinline__ void muon_update(const MuonArgs& p, const MuonJob& J, int64_t at, double x) {
  const float old = J.master != nullptr ? J.master[at] : widen_of(J.param[at], p.f16);
  const float v = static_cast<float>(static_cast<double>(old) * p.decay - J.step * x);
  if (J.master != nullptr) J.master[at] = v;
  J.param[at] = half_of(v, p.f16);
}

// Workgroup: 16 of the long side, wave w the 16-wide tiles w, w + 4, .. of the rank.
__global__ __launch_bounds__(256) void muon_apply_kernel(MuonArgs p, const double* scales, int q_at, int64_t first) {
  int64_t blk = blockIdx.x;
  const bool second = blk >= first;
  const MuonJob& J = job_of(p, first, blk);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane & 15, g = lane >> 4, rp = p.rp;
  const double* Q = J.mat + static_cast<int64_t>(q_at) * rp * rp;
  const double sc = sqrt(scales[second]);
  const int64_t l0 = blk * 16;
  for (int c0 = 16 * wave; c0 < rp; c0 += 64) {
    f64x4 x = {0, 0, 0, 0};
    for (int k0 = 0; k0 < rp; k0 += 4) {
      const int k = k0 + g;
      const double qv = q_at < 0 ? (k == c0 + q ? 1.0 : 0.0) : Q[k * rp + c0 + q];
      if (J.tall)
        x = __builtin_amdgcn_mfma_f64_16x16x4f64(static_cast<double>(J.u[(l0 + q) * rp + k]), qv, x, 0, 0, 0);
      else
        x = __builtin_amdgcn_mfma_f64_16x16x4f64(qv, static_cast<double>(J.u[k * J.len_p + l0 + q]), x, 0, 0, 0);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // tall: long g + 4 e, rank q; wide: rank g + 4 e, long q
      const int64_t l = l0 + (J.tall ? g + 4 * e : q);
      const int c = c0 + (J.tall ? q : g + 4 * e);
      if (l < J.len && c < p.r) muon_update(p, J, J.tall ? l * p.r + c : c * J.len + l, sc * x[e]);
    }
  }
}

// The scales of both matrices, before G is overwritten.
__global__ __launch_bounds__(64) void muon_scale_kernel(MuonArgs p, double* scales) {
  const double s = muon_scale(p.j[blockIdx.x].mat, p.rp, p.eps);
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

struct MuonSizes {
  int64_t len_p, chunk, u, part, mat;
  int chunks;
};
MuonSizes muon_sizes(int64_t len, int64_t r) {
  MuonSizes s;
  const int64_t rp = round_up(r, 16), tiles = cdiv(rp, 64), pairs = tiles * (tiles + 1) / 2;
  s.len_p = round_up(len, 16);
  int64_t chunks = cdiv(96, pairs);
  s.chunk = round_up(cdiv(s.len_p, chunks), 64);
  s.chunks = static_cast<int>(cdiv(s.len_p, s.chunk));
  s.u = align256(s.len_p * rp * 4);
  s.part = align256(static_cast<int64_t>(s.chunks) * pairs * 4096 * 8);
  s.mat = align256(6 * rp * rp * 8);
  return s;
}

}  // namespace

int64_t muon_workspace_bytes(int64_t K, int64_t N, int64_t r) {
  const MuonSizes a = muon_sizes(K, r), b = muon_sizes(N, r);
  return 256 + a.u + a.part + a.mat + b.u + b.part + b.mat;
}

hipError_t launch_muon(int64_t K, int64_t N, int64_t r, uint16_t* A, uint16_t* B, const void* dA, const void* dB,
                       float* mA, float* mB, float* A_master, float* B_master, const qlora_muon_t& o, void* ws,
                       hipStream_t stream, int dtype, bool grad16) {
  MuonArgs p{};
  p.r = static_cast<int>(r);
  p.rp = static_cast<int>(round_up(r, 16));
  p.tiles = (p.rp + 63) / 64;
  p.f16 = dtype == kDtypeF16;
  p.grad16 = grad16;
  p.momentum = o.momentum;
  p.decay = 1.0 - o.lr * o.weight_decay;
  p.nesterov = o.nesterov != 0;
  p.eps = o.eps;
  p.a = o.a;
  p.b = o.b;
  p.c = o.c;
  double* scales = static_cast<double*>(ws);
  char* at = static_cast<char*>(ws) + 256;
  MuonSizes s[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t len = i ? N : K;
    s[i] = muon_sizes(len, r);
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
  const int64_t pairs = static_cast<int64_t>(p.tiles) * (p.tiles + 1) / 2;
  auto grid = [](int64_t a, int64_t b) { return dim3(static_cast<unsigned>(a + b)); };
  Timer tm(QK_MUON, stream);
  const int64_t m0 = cdiv(s[0].len_p * p.rp, 1024), m1 = cdiv(s[1].len_p * p.rp, 1024);
  hipLaunchKernelGGL(muon_momentum_kernel, grid(m0, m1), dim3(256), 0, stream, p, m0);
  hipLaunchKernelGGL(muon_gram_kernel, grid(s[0].chunks * pairs, s[1].chunks * pairs), dim3(256), 0, stream, p, s[0].chunks * pairs);
  hipLaunchKernelGGL(muon_sum_kernel, grid(pairs * 16, pairs * 16), dim3(256), 0, stream, p, pairs * 16);
  hipLaunchKernelGGL(muon_scale_kernel, dim3(2), dim3(64), 0, stream, p, scales);
  const int64_t side = p.rp / 16, wgs = cdiv(side * side, 4);
  for (int i = 0; i < o.steps; ++i)
    for (int what = kSquare; what <= (i + 1 < o.steps ? kNext : kMixed); ++what)
      hipLaunchKernelGGL(muon_product_kernel, grid(wgs, wgs), dim3(256), 0, stream, p, what, i, wgs);
  hipLaunchKernelGGL(muon_apply_kernel, grid(s[0].len_p / 16, s[1].len_p / 16), dim3(256), 0, stream, p,
                     static_cast<const double*>(scales), o.steps == 0 ? -1 : 4 + (o.steps & 1), s[0].len_p / 16);
  tm.stop();
  return hipGetLastError();
}

}  // namespace qn
