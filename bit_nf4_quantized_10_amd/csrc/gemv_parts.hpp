// What the few-row forwards (gemv.hip, mx_gemv.hip) share: the split partials of
// Z = X A beside the base product's, and the launch that adds both up.
#pragma once

#include "common.hpp"
#include "gated.hpp"

namespace qn {

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}

constexpr int kGvWaves = 4;

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// 8 x 8 bf16 transpose: out[t] holds column t of the 8 input rows.
__device__ __forceinline__ void transpose8x8_bf16(const uint4 (&in)[8], uint4 (&out)[8]) {
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const uint32_t sel = (t & 1) ? 0x07060302u : 0x05040100u;
    uint32_t d[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) d[p] = perm(word_of(in[2 * p + 1], t >> 1), word_of(in[2 * p], t >> 1), sel);
    out[t] = make_uint4(d[0], d[1], d[2], d[3]);
  }
}

// Split-K partial of Z = X A for rows row0 .. row0 + 15 over rows [split * 4 rpw, +4 rpw),
// each wave over the rows its GEMV counterpart streams.  A is read row-major
// (8 rows of 8 columns per lane, transposed in registers), X rows feed the
// MFMA as the 16-row operand; lane (q, g) accumulates columns j0 + 8q .. +7.
// The four waves are added in LDS in a fixed order: (w0 + w2) + (w1 + w3).
// zpart[split][m][j], fp32.  red: 16 KB of LDS.
// Inlined by force: as a function it reaches `red` through flat loads, which wait
// for the stores before them (7 us more a call at 8192 x 22016, 1 to 4 rows).
template <class T>
__device__ __forceinline__ void gemv_zpart(const uint16_t* __restrict__ X, int64_t M, int64_t row0, int64_t K, int64_t rpw,
                           const uint16_t* __restrict__ A, int64_t r, float* __restrict__ zpart, int64_t split,
                           float* red) {
  const int t = threadIdx.x, lane = t & 63, q = lane & 15, g = lane >> 4;
  const int wave = t >> 6;
  const int64_t kw0 = (split * kGvWaves + wave) * rpw;
  const int64_t kend = min(K, kw0 + rpw);
  const Rsrc rx = make_rsrc(X, M * K * 2), ra = make_rsrc(A, K * r * 2);
  for (int64_t j0 = 0; j0 < r; j0 += 128) {
    const int64_t j = j0 + 8 * q;
    f32x4 acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = f32x4{0, 0, 0, 0};
    for (int64_t kb = kw0; kb < kend; kb += 32) {
      const int64_t k = kb + 8 * g;
      const uint4 xv =
          ld_b128(rx, (row0 + q < M && k < kend) ? static_cast<uint32_t>(((row0 + q) * K + k) * 2) : kMasked);
      uint4 rows8[8], cols8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        rows8[i] = ld_b128(ra, (k + i < kend && j < r) ? static_cast<uint32_t>(((k + i) * r + j) * 2) : kMasked);
      transpose8x8_bf16(rows8, cols8);
#pragma unroll
      for (int tc = 0; tc < 8; ++tc)
        acc[tc] = T::mfma16(__builtin_bit_cast(typename T::v8, xv), __builtin_bit_cast(typename T::v8, cols8[tc]), acc[tc]);
    }
    // lane holds Z[m = 4g + e][j + tc]
    __syncthreads();
    if (wave >= 2) {
#pragma unroll
      for (int tc = 0; tc < 8; ++tc)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[((wave - 2) * 32 + tc * 4 + e) * 64 + lane] = acc[tc][e];
    }
    __syncthreads();
    if (wave < 2) {
#pragma unroll
      for (int tc = 0; tc < 8; ++tc)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[tc][e] += red[(wave * 32 + tc * 4 + e) * 64 + lane];
    }
    __syncthreads();
    if (wave == 1) {
#pragma unroll
      for (int tc = 0; tc < 8; ++tc)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[(tc * 4 + e) * 64 + lane] = acc[tc][e];
    }
    __syncthreads();
    if (wave == 0 && j < r) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = row0 + 4 * g + e;
        if (m >= M) continue;
        float v[8];
#pragma unroll
        for (int tc = 0; tc < 8; ++tc) v[tc] = acc[tc][e] + red[(tc * 4 + e) * 64 + lane];
        float* o = zpart + (split * M + m) * r + j;
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
}

// Y = sum_s part[s] + c Z B, 16-row tiles.  Workgroup (4 waves) = 512
// columns, row tile blockIdx.y / 4 and its row phase e; lane (q, g) of wave w owns columns
// n0 + 128w + 8q .. +7 and row 4g + e.  A workgroup requests at its start
// the first 8 split partials of its outputs, the first 64 rows of B and the
// first 8 split partials of Z, so that the common case (splits <= 8,
// M r <= 1024, r <= 64) waits for memory once.  The workgroup forms
// Z = RNE_T(sum_s zpart[s]) in LDS, and workgroup (0, 0) writes it out; the
// LoRA product runs on MFMA with Z from LDS and B transposed in registers
// (every phase computes all 16 rows; only row 4g + e is kept).  Partials past
// the last split read as +0 and are added all the same: the running sums
// start at +0 and can never be -0, so adding +0 leaves them unchanged.
constexpr int kFinCols = 512;
__device__ __forceinline__ void fin_add4(float (&s)[4], const uint4 (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s[0] += __builtin_bit_cast(float, v[k].x); s[1] += __builtin_bit_cast(float, v[k].y);
    s[2] += __builtin_bit_cast(float, v[k].z); s[3] += __builtin_bit_cast(float, v[k].w);
  }
}
__device__ __forceinline__ void fin_add8(float (&s)[8], const uint4 (&a)[8], const uint4 (&b)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s[0] += __builtin_bit_cast(float, a[k].x); s[1] += __builtin_bit_cast(float, a[k].y);
    s[2] += __builtin_bit_cast(float, a[k].z); s[3] += __builtin_bit_cast(float, a[k].w);
    s[4] += __builtin_bit_cast(float, b[k].x); s[5] += __builtin_bit_cast(float, b[k].y);
    s[6] += __builtin_bit_cast(float, b[k].z); s[7] += __builtin_bit_cast(float, b[k].w);
  }
}
// kTwo (the gated block; N = F columns per weight, r per member, Z M x 2r): a
// workgroup owns 256 columns, waves 0 and 1 of G, waves 2 and 3 of U; the U
// waves hand their values over in LDS and the G waves store Y = act(G) * U and
// what is kept of G and U.  There Z enters the product in two 16-bit parts, its
// rounding (which is the Z written out) and the rounded rest, within 2^-16 of it
// together: G and U then carry none of Z's rounding, which would move many of their
// 8-bit codes, as above 256 rows.  (One more MFMA a fragment: 0.1 to 0.3 us of the
// 26 of a call at 16 rows, 4096 x 11008, and as much of the 62 at 8192 x 22016.)
template <class T, bool kTwo, bool kGelu>
__global__ __launch_bounds__(256) void gemv_finish_kernel(const float* __restrict__ part, int splits, int64_t M,
                                                          int64_t N, const float* __restrict__ zpart, int zsplits,
                                                          uint16_t* __restrict__ Z, const uint16_t* __restrict__ B,
                                                          int64_t r, float c, uint16_t* __restrict__ Y,
                                                          GatedKeep keep) {
  __shared__ __attribute__((aligned(16))) uint16_t zl[16 * 256];   // Z of 16 rows, 16 x rt (rt <= 256)
  __shared__ __attribute__((aligned(16))) uint16_t zr[kTwo ? 16 * 256 : 8];   // kTwo: the rest of its rounding
  const int t = threadIdx.x, lane = t & 63, q = lane & 15, g = lane >> 4, wave = t >> 6;
  const int e = blockIdx.y & 3;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y >> 2) * 16;
  const int64_t Mt = M - row0 < 16 ? M - row0 : 16;   // rows of this tile
  const int member = kTwo ? wave >> 1 : 0;
  const int64_t ncol = kTwo ? static_cast<int64_t>(blockIdx.x) * (kFinCols / 2) + 128 * (wave & 1) + 8 * q
                            : static_cast<int64_t>(blockIdx.x) * kFinCols + 128 * wave + 8 * q;
  const bool n_ok = ncol < N;
  const int64_t ldn = kTwo ? 2 * N : N, n = ncol + member * N;
  const int64_t rt = kTwo ? 2 * r : r;   // Z's row length
  const int64_t m = row0 + 4 * g + e;
  const bool out_ok = m < M && n_ok;
  const int64_t MR = Mt * rt;            // Z's elements of this tile, from zrow on
  const Rsrc rb = make_rsrc(B, r * ldn * 2);
  const int64_t zrow = row0 * rt, zplane = M * rt;
  const Rsrc rzp = make_rsrc(zpart, static_cast<int64_t>(zsplits) * zplane * 4);
  const Rsrc rp = make_rsrc(part, static_cast<int64_t>(splits) * M * ldn * 4);
  auto load_b = [&](int64_t j0, uint4 (&rows8)[8]) {
    const int64_t jb = j0 + 8 * g;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      rows8[i] = ld_b128(rb, (jb + i < r && n_ok) ? static_cast<uint32_t>(((jb + i) * ldn + n) * 2) : kMasked);
  };
  auto load_part = [&](int s0, uint4 (&pa)[8], uint4 (&pb)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t off = (out_ok && s0 + k < splits) ? static_cast<uint32_t>((((s0 + k) * M + m) * ldn + n) * 4) : kMasked;
      pa[k] = ld_b128(rp, off);
      pb[k] = ld_b128(rp, off == kMasked ? kMasked : off + 16);
    }
  };
  // thread t sums elements idx .. idx+3 of the row-major M x rt matrix Z
  // (rt % 8 == 0, so a group of 4 never leaves its row)
  auto load_z = [&](int s0, int64_t idx, uint4 (&za)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      za[k] = ld_b128(rzp, (idx < MR && s0 + k < zsplits) ? static_cast<uint32_t>(((s0 + k) * zplane + zrow + idx) * 4) : kMasked);
  };
  auto store_z = [&](int64_t idx, const float (&zs)[4]) {
    if (idx >= MR) return;
    const uint2 zv = make_uint2(T::pack2(zs[0], zs[1]), T::pack2(zs[2], zs[3]));
    *reinterpret_cast<uint2*>(zl + idx) = zv;
    if constexpr (kTwo) {
      const uint32_t hi[4] = {zv.x & 0xffffu, zv.x >> 16, zv.y & 0xffffu, zv.y >> 16};
      float rest[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float d = zs[k] - T::widen(hi[k]);
        rest[k] = __builtin_fabsf(d) < __builtin_inff() ? d : 0.0f;   // an infinite rounding has no rest
      }
      *reinterpret_cast<uint2*>(zr + idx) = make_uint2(T::pack2(rest[0], rest[1]), T::pack2(rest[2], rest[3]));
    }
    if (blockIdx.x == 0 && e == 0) *reinterpret_cast<uint2*>(Z + zrow + idx) = zv;
  };
  uint4 pa[8], pb[8], b0[8], b1[8], za[8];
  load_part(0, pa, pb);
  load_b(0, b0);
  load_b(32, b1);
  load_z(0, 4 * t, za);
  {
    float zs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    fin_add4(zs, za);
    for (int s0 = 8; s0 < zsplits; s0 += 8) {
      load_z(s0, 4 * t, za);
      fin_add4(zs, za);
    }
    store_z(4 * t, zs);
  }
  for (int64_t base = 1024; base < MR; base += 1024) {
    float zs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < zsplits; s0 += 8) {
      load_z(s0, base + 4 * t, za);
      fin_add4(zs, za);
    }
    store_z(base + 4 * t, zs);
  }
  __syncthreads();
  f32x4 accl[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) accl[i] = f32x4{0, 0, 0, 0};
  auto lora_step = [&](int64_t j0, const uint4 (&rows8)[8]) {
    const int64_t jb = j0 + 8 * g;
    const int64_t zat = q * rt + member * r + jb;
    const bool z_ok = q < Mt && jb < r;
    const uint4 zv = z_ok ? *reinterpret_cast<const uint4*>(zl + zat) : make_uint4(0, 0, 0, 0);
    uint4 cols8[8];
    transpose8x8_bf16(rows8, cols8);
#pragma unroll
    for (int tc = 0; tc < 8; ++tc)
      accl[tc] = T::mfma16(__builtin_bit_cast(typename T::v8, zv), __builtin_bit_cast(typename T::v8, cols8[tc]), accl[tc]);
    if constexpr (kTwo) {
      const uint4 zd = z_ok ? *reinterpret_cast<const uint4*>(zr + zat) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int tc = 0; tc < 8; ++tc)
        accl[tc] = T::mfma16(__builtin_bit_cast(typename T::v8, zd), __builtin_bit_cast(typename T::v8, cols8[tc]), accl[tc]);
    }
  };
  lora_step(0, b0);
  if (r > 32) lora_step(32, b1);
  for (int64_t j0 = 64; j0 < r; j0 += 32) {
    load_b(j0, b0);
    lora_step(j0, b0);
  }
  if (!kTwo && !out_ok) return;
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  fin_add8(v, pa, pb);
  for (int s0 = 8; s0 < splits; s0 += 8) {
    load_part(s0, pa, pb);
    fin_add8(v, pa, pb);
  }
  if constexpr (kTwo) {
    __shared__ float us[2 * 64 * 9];   // U of the two strips, 8 values a lane (rows of 9: no bank is hit twice)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += c * accl[i][e];
    float* mine = us + ((wave & 1) * 64 + lane) * 9;
    if (member == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[i] = v[i];
    }
    __syncthreads();
    if (member == 1 || !out_ok) return;   // n_ok is the same for the eight lanes of a 64-column block
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = mine[i];
    gated_store8<T, kGelu>(v, u, m, ncol, N, Y, keep);
    return;
  }
  uint4 o;
  o.x = T::pack2(v[0] + c * accl[0][e], v[1] + c * accl[1][e]);
  o.y = T::pack2(v[2] + c * accl[2][e], v[3] + c * accl[3][e]);
  o.z = T::pack2(v[4] + c * accl[4][e], v[5] + c * accl[5][e]);
  o.w = T::pack2(v[6] + c * accl[6][e], v[7] + c * accl[7][e]);
  *reinterpret_cast<uint4*>(Y + m * N + n) = o;
}

}  // namespace

}  // namespace qn
