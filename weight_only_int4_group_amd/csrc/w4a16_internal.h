// Host-side launchers shared between the C-ABI front end and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.h"

namespace w4a16 {

// Bits of the packer's device status word.
constexpr unsigned kPackNonFinite = 1u;
constexpr unsigned kPackRange = 2u;

// Packs row blocks b0 .. b0 + nbw - 1 of the N x K matrix.  rmin/rmax (or
// null for per-group ranges): row n takes entry (n - 16 b0) * rstride.
hipError_t launch_pack(const void *W, const void *s, int N, int K, int b0, int nbw,
                       const uint8_t *keep, const double *rmin, const double *rmax, int rstride,
                       void *Wq, void *scales, void *zeros, unsigned *status, bool symmetric,
                       hipStream_t stream, bool w8 = false);
// Range of W / s (kept weights as 0) of rows n0 .. n0 + rows - 1 into
// rmin/rmax [rows].
hipError_t launch_row_range(const void *W, const void *s, int n0, int rows, int K,
                            const uint8_t *keep, double *rmin, double *rmax, hipStream_t stream);
// acc[0..1] = the least of rmin[0 .. rows) and the largest of rmax, combined
// with acc's earlier value unless `first` (and with 0 always).
hipError_t launch_tensor_range(int rows, const double *rmin, const double *rmax, double *acc,
                               bool first, hipStream_t stream);

// The weights kept in fp16 (validated by the caller): writes row_ptr [N + 1],
// col and val [count], and a keep bit mask in the workspace (returned in
// *mask) for launch_pack.  Blocks until done.  0 on success, -1 on a HIP error.
size_t outlier_workspace_bytes(int N, int K);
int select_outliers(const void *W, const void *s, int N, int K, long long count, int32_t *row_ptr,
                    int32_t *col, _Float16 *val, void *workspace, const uint8_t **mask,
                    hipStream_t stream);

// GPTQ quantize-and-pack (validated by the caller; blocks until done).  0 on
// success, 1 when rocBLAS / rocSOLVER cannot be loaded, 2 when the damped
// Hessian is not positive definite, -1 on a HIP or library error; non-finite
// inputs and scale overflow are flagged in *status as for launch_pack.
size_t gptq_workspace_bytes(int N, int K, long long n);
int gptq_pack(const void *W, const void *s, int N, int K, const void *X, long long n, double damp,
              void *Wq, void *scales, void *zeros, void *workspace, unsigned *status,
              hipStream_t stream);

// One dequantize-matmul problem (validated by the caller).
struct GemmDesc {
  const void *X, *Wq, *scales, *zeros, *s;
  void *Y;
  int M, N, K;
  // optional fp16 outliers, row-compressed (all set or all null)
  const void *o_row_ptr = nullptr, *o_col = nullptr, *o_val = nullptr;
  bool bf16 = false;  // X and Y are bf16 (else fp16)
  bool w8 = false;    // INT8 codes (2048-byte tiles), else INT4
  // streaming path, bf16: workspace for X * s prescaled once per call
  // (skinny_prescale_bytes(M, K) bytes), set by launch_skinny_set
  void *xpre = nullptr;
  // fused epilogue (all or none of a call's problems), or null
  const Fused *fused = nullptr;
  bool gated() const { return fused && fused->gated; }
  int mats() const { return gated() ? 2 : 1; }              // weights of the problem
  int row_blocks() const { return mats() * (N / 16); }      // of all its weights
};

// Streaming kernel for small M (decode and speculative verify): M <= 16.
// launch_skinny_set runs up to skinny_max_problems() independent problems in
// one launch; X * s is staged in K windows when it does not fit in LDS whole,
// or always with force_window.  When the workspace holds
// skinny_workspace_bytes() for the same problems, bf16 problems that run in
// windows get X * s computed once by a small kernel first (else every
// workgroup computes its windows' share itself).
int skinny_max_problems();
size_t skinny_workspace_bytes(const GemmDesc *problems, int count);
hipError_t launch_skinny_set(const GemmDesc *problems, int count, hipStream_t stream,
                             bool force_window = false, void *workspace = nullptr,
                             size_t workspace_bytes = 0);
hipError_t launch_skinny(const void *X, const void *Wq, const void *scales, const void *zeros,
                         const void *s, void *Y, int M, int N, int K, hipStream_t stream);

// LDS-tiled MFMA GEMM for large M (batched decode and prefill): any M >= 1.
// launch_tiled_set runs up to tiled_max_problems() problems in one launch.
// When the workspace holds tiled_workspace_bytes() for the same problems, K
// is split across workgroups where that fills the GPU better (fp32 partials
// in the workspace, then a second launch adds them); otherwise (NULL, or too
// small) every output block walks all of K.
int tiled_max_problems();
size_t tiled_workspace_bytes(const GemmDesc *problems, int count);
hipError_t launch_tiled_set(const GemmDesc *problems, int count, void *workspace,
                            size_t workspace_bytes, hipStream_t stream);
// Adds the split fp32 partials of the fused problems with split > 1 ([M][N] slabs,
// gated [M][2 N]) and applies their epilogues; one activation type per call.
hipError_t launch_fused_reduce(const GemmDesc *const *d, int count, const int *split,
                               float *const *parts, hipStream_t stream);
hipError_t launch_tiled(const void *X, const void *Wq, const void *scales, const void *zeros,
                        const void *s, void *Y, int M, int N, int K, hipStream_t stream);

// Transposed copy of a packed weight for the backward product: codes Wt and
// per-128-row metadata (asynchronous).
hipError_t launch_transpose(const void *Wq, const void *scales, const void *zeros, int N, int K,
                            bool w8, void *Wt, void *meta, hipStream_t stream);

// Gradients of an epilogue: dz = dY * act'(z) and, when u is set, gated: dz =
// dY * u * act'(z), du = dY * act(z).  z null: dz is dY (not written).  db, db2:
// fp32 column sums of dz and du (null: not wanted), which take
// grad_workspace_bytes(M, N, how many) of workspace.
struct GradDesc {
  const void *dY, *z, *u;
  void *dz, *du, *db, *db2;
  int M, N, act;
  bool bf16;
};
size_t grad_workspace_bytes(int M, int N, int sums);
hipError_t launch_grad(const GradDesc &d, void *workspace, hipStream_t stream);

// dX = add + s * sum over the terms of dZ . D (M >= 1, validated by the caller;
// the workspace holds dx_workspace_bytes()).
constexpr int kMaxDxTerms = 4;
struct DxDesc {
  int count;
  const void *dZ[kMaxDxTerms], *Wt[kMaxDxTerms], *meta[kMaxDxTerms];
  int N[kMaxDxTerms];
  const void *s, *add;
  void *dX;
  int M, K;
  bool bf16, w8;
};
size_t dx_workspace_bytes(const DxDesc &d);
hipError_t launch_dx(const DxDesc &d, void *workspace, hipStream_t stream);

// Norms before and after a block: r = alpha x + gate post(y), h = pre(r).  y, gate,
// r and h null where absent; kinds are W4A16_NORM_*.
struct NormSpec {
  int kind;
  float eps;
  const void *weight, *bias;
};
struct NormDesc {
  const void *x, *y, *gate;
  NormSpec post, pre;
  float alpha;
  void *r, *h;
  int T, D, gate_rows;  // gate row m / gate_rows of token m
  bool bf16;
};
hipError_t launch_norm(const NormDesc &d, hipStream_t stream);

// Its backward; sums: the fp32 gradients of the gate, post's weight and bias and
// pre's weight and bias, each null when not wanted.
constexpr int kNormSums = 5;
struct NormGradDesc {
  const void *dr, *dh, *y, *r, *gate;
  NormSpec post, pre;
  float alpha;
  void *dx, *dy;
  void *sums[kNormSums];
  int T, D, gate_rows;
  bool bf16;
};
size_t norm_grad_workspace_bytes(const NormGradDesc &d);
hipError_t launch_norm_grad(const NormGradDesc &d, void *workspace, hipStream_t stream);

// Routing of T tokens to k of E experts (E <= 1024, k <= 64), or its backward (reads
// ids and dweights, writes dlogits).  type: 0 fp16, 1 bf16, 2 fp32 logits.
struct RouteDesc {
  const void *logits;
  const float *bias, *dweights;
  int32_t *ids;
  float *weights;
  void *dlogits;
  int T, E, k, type;
  int sigmoid, groups, topk_groups, renormalize;
  float scale;
};
hipError_t launch_route(const RouteDesc &d, bool grad, hipStream_t stream);

// The experts' gated feed-forward blocks of T tokens with k slots each (validated by the
// caller; D and N multiples of 128, E <= 1024).  A weight holds its E experts one after
// the other: gate and up [N][D], down [D][N].
struct ExpertWeight {
  const void *Wq, *scales, *zeros;
};
struct ExpertsDesc {
  const void *X;
  const int32_t *ids;
  const float *weights;
  ExpertWeight gate, up, down;
  const void *s, *s_down, *residual;
  void *G, *U, *Y;
  int T, E, k, D, N, act;
  bool bf16;
};
size_t experts_workspace_bytes(const ExpertsDesc &d);
hipError_t launch_experts(const ExpertsDesc &d, void *workspace, hipStream_t stream);

// Their backward, from G and U [T][k][N], over the transposed copies of the weights, an
// expert's after the other.  dX and dweights may each be null.
struct ExpertTransposed {
  const void *Wt, *meta;
};
struct ExpertsGradDesc {
  const void *dY;
  const int32_t *ids;
  const float *weights;
  const void *G, *U;
  ExpertTransposed gate, up, down;
  const void *s, *s_down, *add;
  void *dX, *dweights;
  bool dweights_f32;
  int T, E, k, D, N, act;
  bool bf16;
};
size_t experts_grad_workspace_bytes(const ExpertsGradDesc &d);
hipError_t launch_experts_grad(const ExpertsGradDesc &d, void *workspace, hipStream_t stream);

// Speculative-sampling verification of B sequences (validated by the caller):
// the vocabulary is cut into spec_verify_chunks(V) chunks, and the workspace
// (spec_verify_workspace_bytes(B, V) bytes, 256-byte aligned) holds the
// per-chunk sums and the first rejection of every sequence.
int spec_verify_chunks(int V);
size_t spec_verify_workspace_bytes(int B, int V);
hipError_t launch_spec_verify(const float *p_target, const float *p_draft, const int32_t *draft,
                              const float *u_accept, const float *u_sample, int B, int K, int V,
                              void *workspace, int32_t *n_accepted, int32_t *token,
                              hipStream_t stream);

}  // namespace w4a16
