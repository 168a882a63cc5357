// Host-side declarations shared by the kernel translation units and the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qlora_nf4.h"
#include "side_jobs.hpp"

namespace qn {

// Optional per-kernel event timer (see qlora_timer_enable).  Construct right
// before a launch, call stop() right after it; a no-op unless enabled.
// Per-kernel timing for qlora_timer_*: when kernel_id's timer is enabled,
// an event pair brackets the launches between construction and stop().  With
// packet = true the pair is instead handed to one launch through start() /
// end() (hipExtLaunchKernelGGL records it in the dispatch packet itself, so
// it measures that kernel alone); stop() then does nothing.
class Timer {
 public:
  Timer(int kernel_id, hipStream_t stream, bool packet = false);
  void stop();
  hipEvent_t start() const { return static_cast<hipEvent_t>(start_event_); }
  hipEvent_t end() const { return static_cast<hipEvent_t>(packet_stop_); }

 private:
  int id_;
  hipStream_t stream_;
  void* stop_event_;
  void* start_event_;
  void* packet_stop_;
};

// The layer's 16-bit compute type: 0 = bf16, 1 = fp16 (the kDtype of the
// Bf16 / F16 tags); activations, adapters, outputs and the dequantized weight use it.
constexpr int kDtypeBf16 = 0;
constexpr int kDtypeF16 = 1;

// Most member linears in one grouped call (e.g. q, k, v or gate, up).
constexpr int kMaxGroupMembers = 8;

// The read-only view of a stored weight the kernels decode.  With absmax
// non-null the state has no second level: â = absmax[block] (fp32); else
// â = fl32(fl32(fl32(q / 127) * absmax2[block / 256]) + offset).
struct NF4View {
  const uint8_t* codes;
  const int8_t* qabsmax;
  const float* absmax2;
  const float* offset;
  const float* absmax;
};

// A matrix kept as an 8-bit checkpoint (act8.hip): codes rows x cols, absmax
// rows x ceil(cols / 64) in the 16-bit type.  codes null: none given.
struct Act8View {
  const int8_t* codes = nullptr;
  const uint16_t* absmax = nullptr;
};
// ld: row stride of X in elements (a multiple of 8, at least cols).
hipError_t launch_act8_encode(int64_t rows, int64_t cols, const uint16_t* X, int64_t ld, int8_t* codes,
                              uint16_t* absmax, hipStream_t stream, int dtype);
hipError_t launch_act8_decode(int64_t rows, int64_t cols, const int8_t* codes, const uint16_t* absmax, uint16_t* X,
                              int64_t ld, hipStream_t stream, int dtype);

// absmax_out non-null: single-level encoding (the fp32 first-level scales are
// the stored state; qabsmax, absmax2 and offset are not written).
hipError_t launch_quantize(const float* W, int64_t P, uint8_t* codes, int8_t* qabsmax,
                           float* absmax2, float* offset, float* absmax_out, float* ws_absmax, double* ws_gsum,
                           int32_t* ws_flags, int32_t* status, hipStream_t stream);

// ncols != 0: W is K x ncols and goes to columns 0 .. ncols-1 of an output
// with row stride out_ld (ncols a multiple of 8).
hipError_t launch_dequantize(NF4View W, int64_t P, void* out, int out_dtype, int32_t* status, hipStream_t stream,
                             int64_t ncols = 0, int64_t out_ld = 0);

// W' = fl32(ŵ + c A B) (fp64 accumulation; A, B of element type ab_dtype,
// one of NF4_AB_BF16 / NF4_AB_F32 / NF4_AB_F16).
hipError_t launch_merge(int64_t K, int64_t N, int64_t r, NF4View W, const void* A, const void* B, int ab_dtype,
                        float c, float* out, hipStream_t stream);
// One SGD step on A (K x r) and B (r x N) of the 16-bit type dtype,
// optionally through fp32 masters.
hipError_t launch_sgd(int64_t K, int64_t N, int64_t r, uint16_t* A, uint16_t* B, const float* dA, const float* dB,
                      float lr, float* A_master, float* B_master, hipStream_t stream, int dtype = 0);

// A step of A and B along their orthogonalised momentum (muon.hip).
int64_t muon_workspace_bytes(int64_t K, int64_t N, int64_t r);
hipError_t launch_muon(int64_t K, int64_t N, int64_t r, uint16_t* A, uint16_t* B, const void* dA, const void* dB,
                       float* mA, float* mB, float* A_master, float* B_master, const qlora_muon_t& o, void* ws,
                       hipStream_t stream, int dtype, bool grad16);

// Grouped linears sharing X (see layer.hip).
int64_t grouped_fwd_workspace_bytes(int64_t M, int64_t K, int g, const int64_t* Ns, int64_t r);
int64_t grouped_bwd_workspace_bytes(int64_t M, int64_t K, int g, const int64_t* Ns, int64_t r);
hipError_t launch_grouped_fwd(int64_t M, int64_t K, int g, const int64_t* Ns, int64_t r, const uint16_t* X,
                              const NF4View* W, const uint16_t* A, const uint16_t* B, float c, uint16_t* Y,
                              uint16_t* Z, void* ws, hipStream_t stream, int dtype = kDtypeBf16);
hipError_t launch_grouped_bwd(int64_t M, int64_t K, int g, const int64_t* Ns, int64_t r, const uint16_t* G,
                              const uint16_t* X, const uint16_t* Z, const NF4View* W, const uint16_t* A,
                              const uint16_t* B, float c, uint16_t* dX, float* dA, float* dB, void* ws,
                              hipStream_t stream, int dtype = kDtypeBf16);

// Workspace needs (bytes) of the layer kernels; the C ABI adds them up.
int64_t fwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t r);
int64_t bwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t r);

// Split plans of the rank-r products and of the small-M GEMV (sizes in bytes).
struct SkinnyPlan {
  int64_t z_splits, z_per, dz_splits, dz_per, da_splits, da_per, db_splits, db_per;
  int64_t at_bytes, z_part, dz_part, da_part, db_part;
  int64_t gv_rows_per_wave, gv_splits, gv_part, gv_zpart;
};
void plan_gemv(int64_t M, int64_t K, int64_t N, int64_t r, SkinnyPlan* p);
SkinnyPlan plan_skinny(int64_t M, int64_t K, int64_t N, int64_t r);

// The transposes Z = X A needs (Aᵀ into At) and, with cbt != nullptr, the
// forward's LoRA extension operand cbt = RNE_16(c B)ᵀ (N x r).
void lora_transposes(int64_t K, int64_t r, const uint16_t* A, uint16_t* At, int64_t N, const uint16_t* B, float c,
                     uint16_t* cbt, int64_t rb, int dtype, TJob out[2]);
// Z = X A: the transposes above (one launch, unless pre_transposed: another
// launch already ran them), then the split partials and their sum.  z_ext: also
// c Z before its rounding as [hi | lo] (M x 2r, hi + lo to 2^-17).
hipError_t launch_lora_down(int64_t M, int64_t K, int64_t r, const uint16_t* X, const uint16_t* A, uint16_t* Z,
                            const SkinnyPlan& p, void* at_ws, void* part_ws, hipStream_t stream, int64_t N = 0,
                            const uint16_t* B = nullptr, float c = 1.0f, uint16_t* cbt = nullptr, int64_t rb = 0,
                            int dtype = 0, bool pre_transposed = false, uint16_t* z_ext = nullptr);

// Split plans of a group of g linears sharing X (column counts Ns[i], rank r
// each); zp covers Z = X A over all g r columns.
struct GroupPlan {
  SkinnyPlan zp;
  int64_t dz_splits[kMaxGroupMembers], dz_per[kMaxGroupMembers], dz_part, dz_off[kMaxGroupMembers];
  int64_t cs_splits, cs_per, da_part, db_part_total, db_off[kMaxGroupMembers];
};
GroupPlan plan_grouped(int64_t M, int64_t K, int g, const int64_t* Ns, int64_t r);
hipError_t launch_dz_grouped(int64_t M, int g, const int64_t* Ns, int64_t Ntot, int64_t r, const uint16_t* G,
                             const uint16_t* B, float c, uint16_t* dZ, const GroupPlan& gp, void* part_ws,
                             hipStream_t stream, int dtype = 0, RdJob* defer = nullptr, uint16_t* dZ_lo = nullptr);
// dZ_lo (M x g r, or null): what dZ's rounding to 16 bits left out (launch_dz_grouped
// writes it); dA is then formed from both.
hipError_t launch_colsums_grouped(int64_t M, int64_t K, int g, const int64_t* Ns, int64_t Ntot, int64_t r,
                                  const uint16_t* X, const uint16_t* G, const uint16_t* Z, const uint16_t* dZ, float c,
                                  void* dA, void* dB, const GroupPlan& gp, void* da_ws, void* db_ws,
                                  hipStream_t stream, int dtype = 0, bool grad16 = false, Act8View x8 = {},
                                  const uint16_t* dZ_lo = nullptr);
// Small-M forward (M <= 16) in two launches: the split-K partials of X Ŵ and
// of Z = X A (extra workgroups of the same launch), then their fixed-order
// sums, Z (written out) and Y = X Ŵ + c Z B.  part_ws: gv_part + gv_zpart.
hipError_t launch_gemv(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, NF4View W, const uint16_t* A,
                       const uint16_t* B, float c, uint16_t* Y, uint16_t* Z, const SkinnyPlan& p, void* part_ws,
                       hipStream_t stream, int dtype = 0);
// dZ = c G Bᵀ: split partials, then their sum (with defer != nullptr that sum
// is not launched but returned, for the caller to run in a later launch).
// dZ_lo (M x r, may be null): what dZ's rounding leaves out, in 16 bits.
hipError_t launch_dz(int64_t M, int64_t N, int64_t r, const uint16_t* G, const uint16_t* B, float c, uint16_t* dZ,
                     const SkinnyPlan& p, void* part_ws, hipStream_t stream, int dtype = 0, RdJob* defer = nullptr,
                     uint16_t* dZ_lo = nullptr);
// dA and dB: fp32, or with grad16 of the layer's 16-bit type.  x8 (codes
// non-null): X is kept in 8 bits, and the X argument is not read.  dZ_lo (may be
// null): dA = Xᵀ (dZ + dZ_lo).
hipError_t launch_colsums(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, const uint16_t* G,
                          const uint16_t* Z, const uint16_t* dZ, float c, void* dA, void* dB, const SkinnyPlan& p,
                          void* da_ws, void* db_ws, hipStream_t stream, int dtype = 0, bool grad16 = false,
                          Act8View x8 = {}, const uint16_t* dZ_lo = nullptr);

hipError_t launch_fwd(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, NF4View W,
                      const uint16_t* A, const uint16_t* B, float c, uint16_t* Y, uint16_t* Z,
                      void* ws, hipStream_t stream, int dtype = 0);

hipError_t launch_bwd(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G,
                      const uint16_t* X, const uint16_t* Z, NF4View W, const uint16_t* A,
                      const uint16_t* B, float c, uint16_t* dX, void* dA, void* dB, void* ws,
                      hipStream_t stream, int dtype = 0, bool grad16 = false, Act8View x8 = {});

// Split-K plan of the 256 x 256-tile GEMMs for an M x cols output reduced
// over red: splits (1: none), elements per split, fp32 partial bytes.
struct SplitPlan {
  int64_t splits, k_per, part_bytes;
};
SplitPlan plan_split(int64_t M, int64_t cols, int64_t red);
// out = the 16-bit rounding of the sum of `splits` fp32 planes of count
// elements (count % 8 == 0) in order.
hipError_t launch_split_sum(const float* part, int64_t splits, int64_t count, uint16_t* out, hipStream_t stream,
                            int dtype);

// The GEMMs below split their reduction per plan_split when split_ws (at
// least part_bytes, 16-byte aligned) is given, then sum the partials in
// split order into the 16-bit output (a second launch).
// cBt: RNE_bf16(c B)ᵀ, N x r
hipError_t launch_fwd_big(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, NF4View W,
                          const uint16_t* Z, const uint16_t* cBt, uint16_t* Y, hipStream_t stream, int dtype = 0,
                          void* split_ws = nullptr);

hipError_t launch_dx_big(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, NF4View W,
                         const uint16_t* dZ, const uint16_t* A, uint16_t* dX, hipStream_t stream, int dtype = 0,
                         void* split_ws = nullptr);

hipError_t launch_fwd_dense(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, const uint16_t* WhatT,
                            const uint16_t* Z, const uint16_t* cBt, uint16_t* Y, hipStream_t stream, int dtype = 0,
                            void* split_ws = nullptr);
// Forward over g members' concatenated columns (Ntot in all, member i ending
// at column gend[i], every member a multiple of 256 columns): Zcat is M x g r,
// member i's Z in columns i r .. +r; WhatT and cBt are the members' Ŵᵀ and
// (c B)ᵀ stacked row-wise (Ntot x K and Ntot x r).
hipError_t launch_fwd_dense_grouped(int64_t M, int64_t K, int64_t Ntot, int64_t r, const uint16_t* X,
                                    const uint16_t* WhatT, const uint16_t* Zcat, int g, const int64_t* gend,
                                    const uint16_t* cBt, uint16_t* Y, hipStream_t stream, int dtype = 0,
                                    void* split_ws = nullptr);
hipError_t launch_dx_dense(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, const uint16_t* What,
                           const uint16_t* dZ, const uint16_t* A, uint16_t* dX, hipStream_t stream, int dtype = 0,
                           void* split_ws = nullptr);

// The gated feed-forward front (gated.hip; up to 256 rows gemv.hip): W[0], W[1]
// the K x F weights, A K x 2r, B r x 2F, H M x F (null in launch_gated_dense:
// not wanted), Z M x 2r.
struct GatedKeep;
int64_t gated_fwd_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t r);
int64_t gated_bwd_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t r);
hipError_t launch_gated_fwd(int64_t M, int64_t K, int64_t F, int64_t r, const uint16_t* X, const NF4View* W,
                            const uint16_t* A, const uint16_t* B, float c, bool gelu, uint16_t* H, uint16_t* Z,
                            const GatedKeep& keep, void* ws, hipStream_t stream, int dtype);
// kept: the forward's; with neither kept, G and U are computed again from X.
hipError_t launch_gated_bwd(int64_t M, int64_t K, int64_t F, int64_t r, const uint16_t* dH, const uint16_t* X,
                            Act8View x8, const uint16_t* Z, const GatedKeep& kept, const NF4View* W, const uint16_t* A,
                            const uint16_t* B, float c, bool gelu, uint16_t* dX, void* dA, void* dB, void* ws,
                            hipStream_t stream, int dtype, bool grad16);
SplitPlan plan_split16(int64_t M, int64_t cols, int64_t red);
// Columns of the split (from `first` on; first = F and one split: none) and its parts.
struct GatedSplit {
  int64_t first, splits, k_per, part_bytes;
};
GatedSplit plan_gated_split(int64_t M, int64_t K, int64_t F);
// w_ld: row stride of WhatT.
hipError_t launch_gated_dense(int64_t M, int64_t K, int64_t F, int64_t r, const uint16_t* X, const uint16_t* WhatT,
                              int64_t w_ld, const uint16_t* Zext, const uint16_t* Bt, bool gelu, uint16_t* H, const GatedKeep& keep,
                              hipStream_t stream, int dtype, void* split_ws);
// dX = dY Ŵᵀ + dZ Aᵀ: dY M x red, What K x red, dZ M x rt, A K x rt.
hipError_t launch_gated_dx(int64_t M, int64_t K, int64_t red, int64_t rt, const uint16_t* dY, const uint16_t* What,
                           const uint16_t* dZ, const uint16_t* A, uint16_t* dX, hipStream_t stream, int dtype,
                           void* split_ws);
hipError_t launch_gated_dy(int64_t M, int64_t F, const uint16_t* dH, const GatedKeep& kept, bool gelu, uint16_t* dY,
                           hipStream_t stream, int dtype);
// Up to 256 rows: split-K partials of both weights and of Z, then their sums.
struct GatedGemvPlan {
  int64_t rows_per_wave, splits, part, zpart;
};
GatedGemvPlan plan_gated_gemv(int64_t M, int64_t K, int64_t F, int64_t r);
hipError_t launch_gated_gemv(int64_t M, int64_t K, int64_t F, int64_t r, const uint16_t* X, const NF4View* W,
                             const uint16_t* A, const uint16_t* B, float c, bool gelu, uint16_t* H, uint16_t* Z,
                             const GatedKeep& keep, void* ws, hipStream_t stream, int dtype);

// The output head's cross entropy (head.hip): X M x K, W V x K, dX null: the
// loss alone; lse may be null.
int64_t head_workspace_bytes(int64_t M, int64_t K, int64_t V, bool need_dx);
hipError_t launch_head_loss(int64_t M, int64_t K, int64_t V, const uint16_t* X, const uint16_t* W, const int64_t* targets,
                            const float* weights, int64_t ignore, float* loss, float* lse, uint16_t* dX, void* ws,
                            hipStream_t stream, int dtype);

// A matrix held in MXFP4 (mxfp4.hpp has its layout).
struct MxView {
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, cols;
};
// type: of X, one of NF4_OUT_*.  across: X is cols x rows.  ld: X's row stride.
hipError_t launch_mx_quantize(int type, bool across, const void* X, int64_t ld, MxView m, hipStream_t stream);
hipError_t launch_mx_dequantize(int type, bool across, MxView m, void* X, int64_t ld, hipStream_t stream);
// Products for fewer rows than tiles want (mx_gemv.hip): which kernel, tiles of 16 act and
// weight rows a wave, splits of the reduction and the bytes of their fp32 planes (0: the
// output is written itself), and the same of Z = X A.
enum { kMxDecode, kMxRows, kMxPanel };
struct MxRowsPlan {
  int kind, ra, rw;
  int64_t splits, chunks_per, part;
  int64_t zsplits, z_rpw, zpart;
};
MxRowsPlan plan_mx_rows(int64_t M, int64_t K, int64_t N, int64_t r);
// Quantises X (M x K) into m; in the same launch Z's partials (pl given) or two transposes.
hipError_t launch_mx_front(MxView m, const uint16_t* X, hipStream_t stream, int dtype, const MxRowsPlan* pl, const uint16_t* A, int64_t r,
                           float* zpart, const TJob* side);
// kMxDecode takes X and quantises it on the way, with Z's partials, the others act.  out:
// planes, or with one split the output in 16 bits (out16) or 32.
hipError_t launch_mx_rows(const MxRowsPlan& pl, const uint16_t* X, const MxView* act, MxView w, int64_t M, void* out, bool out16,
                          hipStream_t stream, int dtype, const uint16_t* A = nullptr, int64_t r = 0, float* zpart = nullptr);
// Z and Y = the planes' sum + c Z B.
hipError_t launch_mx_rows_finish(const MxRowsPlan& pl, const float* part, const float* zpart, int64_t M, int64_t N, int64_t r,
                                 const uint16_t* B, float c, uint16_t* Y, uint16_t* Z, hipStream_t stream, int dtype);
// dX by a product that decodes W itself (mx_back.hip).  splits 0: W is dequantised, and the
// product dense; else ranges of the reduction, rows of W each, and their planes' bytes.
struct MxBackPlan {
  int64_t splits, per, part;
};
MxBackPlan plan_mx_back(int64_t M, int64_t K, int64_t N);
hipError_t launch_mx_back(const MxBackPlan& pl, int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, const uint16_t* dZ,
                          MxView W, const uint16_t* A, uint16_t* dX, float* part, hipStream_t stream, int dtype);
// out (p.rows x q.rows, of out_type) = p qᵀ
int64_t mx_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_matmul(MxView p, MxView q, int out_type, void* out, void* ws, hipStream_t stream);
// The layer on an MXFP4 weight W (N x K).
int64_t mx_fwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t r);
int64_t mx_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t r);
hipError_t launch_mx_fwd(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* X, MxView W, const uint16_t* A,
                         const uint16_t* B, float c, uint16_t* Y, uint16_t* Z, void* ws, hipStream_t stream, int dtype);
hipError_t launch_mx_bwd(int64_t M, int64_t K, int64_t N, int64_t r, const uint16_t* G, const uint16_t* X, Act8View x8,
                         const uint16_t* Z, MxView W, const uint16_t* A, const uint16_t* B, float c, uint16_t* dX,
                         void* dA, void* dB, void* ws, hipStream_t stream, int dtype, bool grad16);

// Dequantize a K x N weight to the 16-bit compute type (dtype), either as
// stored (K x N) or transposed (N x K).
// out_ld: row stride of the output (0: N, transposed K).
// Side jobs run as extra workgroups of the same launch: side_t (two
// transposes, transposed output only), side_r (one split sum, untransposed
// output only).
hipError_t launch_dequant_bf16(NF4View W, int64_t K, int64_t N, bool transposed, uint16_t* out, hipStream_t stream,
                               int64_t out_ld = 0, int dtype = 0, const TJob* side_t = nullptr,
                               const RdJob* side_r = nullptr);

}  // namespace qn
