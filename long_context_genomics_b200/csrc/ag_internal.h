// ag_internal.h -- launchers shared between the C-ABI layer and the kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/ag.h"

namespace ag {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType,
                                   cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

// Scratch of the attention kernel's range schedule (ag_attn_fwd_noalloc) for
// pairs of query tiles whose key range is split between clusters: per slot a
// partial output [2][128][Dv] fp32 (sized for the widest Dv, 192) and a
// partial log-sum-exp [2][128] fp32.  Nothing in it must be initialised.
constexpr size_t kAttnSlotOutBytes = 2 * 128 * 192 * sizeof(float);
constexpr size_t kAttnSlotLseBytes = 2 * 128 * sizeof(float);
inline size_t attn_scratch_bytes(int slots) {
  return static_cast<size_t>(slots) * (kAttnSlotOutBytes + kAttnSlotLseBytes);
}

// Keys per K/V tile of the attention kernel, and its work steps: pairs of
// 128-row query tiles (16 positions x 8 heads each) times key tiles.  The
// kernel indexes steps with int, so callers keep this at or below 2^30.
constexpr int64_t kAttnKeyTile = 128;
// Most 2-CTA clusters an attention launch uses (one per SM pair up to 256 SMs).
constexpr int kAttnMaxClusters = 128;
inline int64_t attn_work_steps(int64_t B, int64_t Lq, int64_t L) {
  const int64_t blocks = (Lq + 15) / 16;  // the last may be partial
  return B * ((blocks + 1) / 2) * ((L + kAttnKeyTile - 1) / kAttnKeyTile);
}
inline int64_t attn_work_steps(int64_t B, int64_t L) { return attn_work_steps(B, L, L); }

struct AttnLaunch {
  const void *q, *k, *v;
  const float *bias;
  int64_t bias_bstride;  // floats between batch items' bias (0: shared)
  float *out, *lse;
  int64_t B, L;         // batch items, keys per item
  int64_t Lq;           // query positions per item (rows of q, out and lse)
  int64_t Dv;           // value width: 128 or 192
  float cap;
  unsigned *err;        // device error word
  int num_sms;
  void *scratch;        // NULL: schedules that need no scratch (whole pairs or
                        // two launches); else attn_scratch_bytes(scratch_slots)
                        // bytes, 256-aligned, for the range schedule
  int scratch_slots;    // clusters the range schedule may use (>= 1)
  EncodeTiledFn encode;
  cudaStream_t stream;
};

// Returns cudaSuccess or the first CUDA error; CUDA_ERROR_* from tensor-map
// encoding is reported as cudaErrorInvalidValue.
cudaError_t launch_attn_fwd(const AttnLaunch &a);

// How many kernels launch_attn_fwd launches for these sizes on the current
// device (0 for an empty call, 1, or 2 when split pairs need the merge kernel
// or a second launch); scratch_slots 0 for the schedules without scratch.
cudaError_t attn_fwd_kernel_count(int64_t B, int64_t Lq, int64_t L, int64_t Dv, float cap,
                                  int num_sms, int scratch_slots, int *count);
// The schedule launch_attn_fwd uses for these sizes with sm_pairs resident
// 2-CTA clusters (pure host logic): wb and fb hold kAttnMaxClusters + 1 ints.
void attn_fwd_schedule(int64_t B, int64_t L, int sm_pairs, int scratch_slots, int *sched,
                       int *clusters, int *tail_clusters, int *whole, int *n_whole,
                       int *split_at, int *wb, int *fb);
// How many 2-CTA clusters the first launch of such a call uses.
cudaError_t attn_fwd_clusters(int64_t B, int64_t L, int64_t Dv, float cap, int num_sms,
                              int scratch_slots, int *clusters);

// Backward of the attention (attn_bwd.cu): two kernels, the query kernel
// (delta, dq) then the key kernel (dk, dv, dbias), on `stream`.
struct AttnBwdLaunch {
  const void *q, *k, *v;  // bf16 [B,H,L,128], [B,L,128], [B,L,Dv]
  const float *bias;
  int64_t bias_bstride;   // floats between batch items' bias (0: shared)
  const float *lse, *dout;
  float *delta, *dq, *dk, *dv, *dbias;
  int64_t B, H, L, Dv;
  float cap;              // > 0, +inf for no cap
  cudaStream_t stream;
};
cudaError_t launch_attn_bwd(const AttnBwdLaunch &a);
int attn_bwd_kernel_count();
// Tensor-core backward (attn_bwd_sm100.cu): value width 128, q, k, v, dout
// and dq 16-byte aligned; four launches (dout split, query pass 1, key pass,
// query pass 2).  Uses dq as the staging place of dout's bf16 halves.
bool attn_bwd_tc_supported(const AttnBwdLaunch &a);
cudaError_t launch_attn_bwd_tc(const AttnBwdLaunch &a, int num_sms, unsigned *err,
                               EncodeTiledFn encode);

// Projects `cells` consecutive cells of 128 channels into 8 head planes of
// `cells` floats each.
cudaError_t launch_pair_bias_project(const float *pair, const float *W,
                                     float *bias, int64_t cells, int num_sms,
                                     unsigned *err, EncodeTiledFn encode,
                                     cudaStream_t stream);

// Linear layers (linear.cu, linear_sm100.cu): what is done to a product's
// float32 sums before they are stored (linear_epilogue.cuh).
struct LinearEpilogue {
  const float *bias;      // [columns], or NULL
  const void *pre_in;     // multiply by act'(pre_in), or NULL: apply act
  void *pre_out;          // the sums with their bias, rounded to dtype, or NULL
  const void *residual;   // of the output's type, or NULL
  void *out;
  int64_t ld_pre_in, ld_pre_out, ld_res, ld_out;
  int act, dtype, out_dtype;  // dtype: of the operands, pre_in and pre_out
  int vec8;               // rows of 8-column groups are 16-byte aligned in every array
};
struct LinearFwd {
  const void *x, *W;
  int64_t ldx, ldw, M, N, K;
  LinearEpilogue epi;
  void *workspace;
  int num_sms;
  unsigned *err;
  EncodeTiledFn encode;
  cudaStream_t stream;
};
cudaError_t linear_fwd_workspace(const LinearFwd &a, int64_t *bytes);
cudaError_t launch_linear_fwd(const LinearFwd &a);
struct LinearBwd {
  const void *dy, *x, *W;
  int64_t lddy, ldx, ldw, M, N, K;
  LinearEpilogue dx, dW;  // out NULL: not wanted
  float *db;              // or NULL
  void *workspace;
  int num_sms;
  unsigned *err;
  EncodeTiledFn encode;
  cudaStream_t stream;
};
cudaError_t linear_bwd_workspace(const LinearBwd &a, int64_t *bytes);
cudaError_t launch_linear_bwd(const LinearBwd &a);

// Norm and rotation of queries and keys (qk_norm_rope.cu).
struct QkSide {
  const void *x;          // [B, L, H, D] with element strides sb, sl, sh
  int64_t sb, sl, sh;
  int H;
  const float *w, *b;
  void *out;              // forward: [B, H, L, D]
  const void *g;          // backward: upstream gradient [B, H, L, D]
  void *dx;               // backward: element strides db_, dl, dh
  int64_t dxb, dxl, dxh;
  float *dw, *db;         // backward: parameter gradients, or NULL
};
struct QkArgs {
  QkSide side[2];         // queries, keys
  const double *inv_freq;
  const int64_t *positions;
  int64_t pos_sb;
  int64_t positions_total;  // B * L
  int64_t B, L;
  int D, R, norm, rope, x_dtype, o_dtype;  // o_dtype: of out or g
  float eps;
  float *partial;         // backward: parameter gradients' partial sums
};
cudaError_t launch_qk_fwd(const QkArgs &a, int num_sms, cudaStream_t stream);
cudaError_t launch_qk_bwd(const QkArgs &a, int num_sms, cudaStream_t stream);
int64_t qk_bwd_workspace(int64_t positions_total, int Hq, int Hk, int D, int num_sms);

// Global gradient norm and clipping (grad_clip.cu).
cudaError_t launch_grad_clip(void *const *grads, const int64_t *counts, const int *dtypes,
                             int64_t n, float max_norm, float eps, float *norm_out,
                             double *workspace, int num_sms, cudaStream_t stream);
int64_t grad_clip_workspace(int64_t n, int num_sms);

cudaError_t launch_wait_timeout_probe(uint64_t timeout_ns, unsigned *err,
                                      cudaStream_t stream);

// Shared by the entry points (ag_api.cu).
struct DeviceInfo {
  bool ready = false;
  bool sm100 = false;
  int num_sms = 0;
  unsigned *err = nullptr;  // device address of the device error word
};
// Per-device set-up of the current device, done once; AG_ERR_UNSUPPORTED on
// anything but sm_100.
ag_status device_info(DeviceInfo **out);
ag_status get_encoder(EncodeTiledFn *fn);
ag_status check_attn_sizes(int64_t B, int64_t H, int64_t L, int64_t D, int64_t block,
                           float cap);
bool aligned(const void *p, uintptr_t a);
bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb);
ag_status from_cuda(cudaError_t e);

}  // namespace ag
