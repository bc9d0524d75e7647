// Host-side descriptions of the layer operators' kernel calls (linear
// attention, block norm, gradient clipping), shared by their C entry points
// (ssd_layer_api.cu) and the kernel launchers.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// One operand [B][T][heads][D]: the last two dimensions are dense, the others
// have strides (in elements); head h of the walk reads head h / share.
struct LaOperand {
  const void* p;
  long long batch, step;
  int share;
};

// One walk over the steps of every (b, h): with a = e^{log_decay[h]} and the
// steps of a row of length n taken in order (or from the last one back),
//   o_i    = s_intra sum_{j <= i} a^{i-j} (q_i . k_j) v_j + s_carry a^{i+off} first q_i
//   last   = a^n first + s_inject sum_j a^{n-1-j + (1-off)} v_j k_j^T
// (i, j count in the order of the walk).  The forward is one walk; dq, dk and
// dv are walks with the operands' roles exchanged, the last two backwards.
struct LaWalk {
  int B, T, H, dk, dv;
  LaOperand q, k, v;
  const float* log_decay;
  const float* first;     // [B][H][dv][dk], or [B][H][dk][dv] if swapped; nullable
  float* last;            // same layout; nullable
  bool first_swapped;
  const int* lens;        // [B], nullable
  void* o;                // [B][T][H][dv], dense
  float s_intra, s_carry, s_inject;
  int off;
  bool reverse;
  bool followed;          // the next launch on the stream is a walk `beside` this one
  void* hist;             // bf16 walks: the states before every chunk (la_tc_hist_rows rows of
                          // 64), nullable; with it o may be NULL (the states alone)
};

// SMs of the GPU that the library is built for.  A constant, so that the
// segments that a row is cut into, and with them the workspace's size and the
// order of the sums, are the same wherever they are asked for (without a GPU too).
constexpr int kLaSms = 152;

// scratch: la_scratch_floats() floats
size_t la_scratch_floats(int B, int H, int T, int dk, int dv, bool bf16);
// `beside`: the walk needs nothing of the kernel launched before it, which is
// another walk, and may run beside it.
cudaError_t la_walk(const LaWalk& w, bool bf16, bool beside, float* scratch, cudaStream_t s);
// Segments of a row that is shared out over CTAs, `slots` of which run at once.
int la_segments(long long rows, long long chunks, long long slots);
// the states before each segment from the segments' own states (in place)
struct LaSegments {
  int B, H, T, dk, dv, nseg, span;  // span: steps of a segment
  const float* log_decay;
  const int* lens;
  float* seg;          // [nseg][B][H][dv][dk]
  const float* first;  // nullable; [dk][dv] instead of [dv][dk] if swapped
  float* last;         // nullable
  bool swapped, reverse;
};
cudaError_t la_segment_states(const LaSegments& p, cudaStream_t s);
// the bf16 walk on tensor cores (ssd_linattn_tc.cu)
size_t la_tc_scratch_floats(int B, int H, int T, int dk, int dv);
cudaError_t la_walk_tc(const LaWalk& w, bool beside, float* scratch, cudaStream_t s);
// dq and dk from the states before every chunk, forward and backward, summed
// over the heads that share them (every bf16 backward)
struct LaGrads {
  int B, T, H, dk, dv;
  LaOperand q, k, v, dout;
  const float* log_decay;
  const int* lens;
  const void *hist_s, *hist_g;
  void *dq, *dk_out;
  float scale;
};
long long la_tc_hist_rows(int B, int H, int T, int dk, int dv);
cudaError_t la_grads_tc(const LaGrads& d, cudaStream_t s);
// reads and clears the kernels' device error word (a wait gave up)
cudaError_t la_read_and_clear_error(unsigned int* out);
// a CTA whose bounded wait runs out
cudaError_t la_selftest_timeout(cudaStream_t s);
// out[b][t][g][:] = sum over the group's heads of part[b][t][h][:], in head
// order (fp32)
cudaError_t la_group_sum(long long rows, int G, int share, int D, const float* part, float* out,
                         cudaStream_t s);

struct LaStep {
  int B, H, G, dk, dv;
  const void *q, *k, *v;
  long long q_batch, k_batch, v_batch;
  const float* log_decay;
  long long decay_batch;  // 0, or H: a decay for each row too
  const float* state_in;
  float* state_out;
  const int* slots;       // [B] rows of the state, nullable
  long long nslots;
  void* o;
  float scale;
};
cudaError_t la_step(const LaStep& p, bool bf16, cudaStream_t s);

// The gated delta rule (ssd_delta.cu, ssd_delta_grads.cu).  Rows are walked in
// chunks of delta_chunk() steps; the backward keeps, for every row and head and
// each of the row's chunks, the state before it and the gradient of the state
// after it [dv][dk], and E and y [steps][dv], all fp32.
int delta_chunk(bool bf16);
struct DeltaWalk {
  int B, T, H, dk, dv;
  LaOperand q, k, v;
  const float *log_decay, *beta;  // [B][T][H]
  const float* first;             // [B][H][dv][dk], nullable
  float* last;                    // nullable
  const int* lens;
  void* o;
  float *hist, *err;              // given: the states before every chunk and E instead of o
  float scale;
};
cudaError_t delta_walk(const DeltaWalk& p, bool bf16, cudaStream_t s);
struct DeltaBack {
  int B, T, H, dk, dv;
  LaOperand q, k, dout;
  const float *log_decay, *beta;
  const float* first;  // gradient of the final state, nullable
  float* last;         // of the first one, nullable
  const int* lens;
  void* dv_out;
  float *hist, *y;
  float scale;
};
cudaError_t delta_back(const DeltaBack& p, bool bf16, cudaStream_t s);
struct DeltaGrads {
  int B, T, H, G, dk, dv;
  LaOperand q, k, dout;
  const float *log_decay, *beta;
  const int* lens;
  const float *hist_s, *hist_d, *err, *y;
  void *dq, *dk_out;
  float *dlog_decay, *dbeta;
  float scale;
};
// part: for heads that share q and k, 2 B T H dk floats
cudaError_t delta_grads(const DeltaGrads& p, float* part, bool bf16, cudaStream_t s);
struct DeltaStep {
  int B, H, G, dk, dv;
  const void *q, *k, *v;
  long long q_batch, k_batch, v_batch;
  const float *log_decay, *beta;  // [B][H]
  const float* state_in;
  float* state_out;
  const int* slots;  // nullable
  long long nslots;
  void* o;
  float scale;
};
cudaError_t delta_step(const DeltaStep& p, bool bf16, cudaStream_t s);

// Norms around a block (ssd_blocknorm.cu).  In the backward `residual` is the
// forward's new residual.  part: [grid][2][width] column sums of the CTAs,
// grid <= kBlockNormMaxCtas.
constexpr int kBlockNormMaxCtas = 608;
struct BlockNorm {
  long long rows;
  int width;
  long long y_stride, z_stride;
  float eps;
  const void *residual, *y, *z;
  const float *w_post, *res_scale, *w_pre;
  void *new_residual, *x;
  float* stats;
  const void *dx, *dnew;
  void *dresidual, *dy, *dz;
  float *dw_post, *dres_scale, *dw_pre;
  float* part;
};
cudaError_t block_norm_forward(const BlockNorm& p, bool bf16, bool res_bf16, cudaStream_t s);
cudaError_t block_norm_backward(const BlockNorm& p, bool bf16, bool res_bf16, cudaStream_t s);

// Layer norm (ssd_layernorm.cu).  part: [grid][2][width] column sums of the CTAs,
// grid <= kLayerNormMaxCtas.
constexpr int kLayerNormMaxCtas = 608;
struct LayerNorm {
  long long rows;
  int width;
  long long x_stride;
  float eps;
  const void* x;
  const float *weight, *bias;  // nullable
  void* y;
  float* stats;  // [rows][2] mean, 1 / sqrt(variance + eps); nullable
  const void* dy;
  void* dx;
  float *dweight, *dbias;  // nullable
  float* part;
};
cudaError_t layer_norm_forward(const LayerNorm& p, bool bf16, cudaStream_t s);
cudaError_t layer_norm_backward(const LayerNorm& p, bool bf16, cudaStream_t s);

// Gradient clipping (ssd_clip.cu): `count` tensors, none empty, cut into
// chunks of 2^shift bytes; kClipTable tensors a launch, at most kClipMaxCtas
// partial sums each.
constexpr int kClipTable = 960;
constexpr int kClipMaxCtas = 1216;
struct ClipEntry {
  const void* g;
  void* out;
  long long numel;
  int first_chunk;  // set by the launcher
  int bf16;
};
cudaError_t clip_grad_norm(const ClipEntry* e, int count, int shift, double* part, float max_norm,
                           float eps, float* norm, cudaStream_t s);

// The calling thread's last-error message (ssd_api.cu).
void set_last_error(const char* msg);

}  // namespace ssd
