/*
 * kda_layer.h -- C ABI of the operators that stand around the KDA recurrence in a
 * layer: the short causal convolution before it, the selective state space scan as
 * its sibling token mixer, and the norms before and after a block.  The conventions
 * of kda.h hold (device pointers, caller-owned buffers, nothing allocated or
 * synchronised, work enqueued on `stream` only, errors as kda_status before
 * anything is enqueued, no implicit conversion), and every entry point can be
 * captured into a CUDA graph.
 *
 * Rows.  Activations are rows of one type, bf16 or fp32 (kda_row_dtype), [B, T, C]
 * with contiguous channels.  An argument `*_stride` is the distance, in elements,
 * between two tokens' rows, so that a part of a wider projection is read in place;
 * sequence b starts at token b * T.  Buffers without a stride argument are
 * contiguous.  Any alignment of the element type is accepted; 16-byte aligned
 * rows (pointer, stride and channel count) take the vector path.
 * Parameters (weights, biases, A_log, ...) and their gradients are fp32; sums,
 * states and norms are held in fp32.
 *
 * Sequences.  cu_seqlens as in kda_fwd: NULL (batched), or int64 [N+1] on the
 * device with B == 1, cu[0] = 0, non-decreasing, cu[N] <= T; rows from cu[N] on
 * belong to no sequence: their values count for nothing, outputs are left as they were
 * there, and a backward writes zeros as their gradients.  Empty sequences are allowed:
 * their final state is their initial one.
 * An inconsistent cu_seqlens is recorded as KDA_ERR_BAD_SEQLENS in the workspace's
 * status word (kda_get_device_status); the tokens it misplaces are skipped or
 * computed from a wrong start, and no access leaves the buffers.
 * Results are bitwise identical run to run: every sum has a fixed order.
 */
#ifndef KDA_LAYER_H_
#define KDA_LAYER_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Storage type of activation rows. */
typedef enum { KDA_ROW_BF16 = 0, KDA_ROW_FP32 = 1 } kda_row_dtype;

/* Elementwise function: of the convolution (NONE, SILU) and of a norm's gate. */
typedef enum { KDA_FN_NONE = 0, KDA_FN_SILU = 1, KDA_FN_SIGMOID = 2 } kda_fn;

#define KDA_CONV_MAX_WIDTH 4
#define KDA_CONV_MAX_OUTS 4
#define KDA_NORM_MAX_DIM 8192
#define KDA_SCAN_CHUNK 32       /* tokens between two saved states of the scan */
#define KDA_STATUS_BYTES 256    /* a workspace that holds a status word only    */

/* ----------------------------------------------------------- convolution --
 * kda_conv_fwd -- causal depthwise convolution over each sequence, with its
 * activation:
 *     p[t][c]   = bias[c] + sum_{j < width} weight[c][j] * xx[t - width + 1 + j][c]
 *     out[t][c] = fn(p[t][c])
 * where xx is the sequence's x with the width - 1 rows of its initial state before
 * it (zeros when initial_state is NULL).  The final state is the last width - 1
 * rows of xx.  One token at a time is the case T == 1 with the states carried, which has
 * a kernel of its own; single tokens packed with cu_seqlens do not reach it.
 *   x               rows [B, T, C], x_stride.
 *   weight          fp32 [C, width]; bias fp32 [C] or NULL (zero).
 *   outs            num_outs (1 .. KDA_CONV_MAX_OUTS) host array of device buffers;
 *                   outs[i] is [B, T, out_channels[i]] and receives the next
 *                   out_channels[i] channels (q, k and v of one projection); the
 *                   counts are positive and sum to C.
 *   initial_state   NULL or [N, width - 1, C] of the rows' type.
 *   final_state     NULL or the same shape, written; it may be initial_state itself.
 *   width           2 .. KDA_CONV_MAX_WIDTH.     fn  KDA_FN_NONE or KDA_FN_SILU.
 *   workspace       NULL, or a device buffer (128-byte aligned, KDA_STATUS_BYTES)
 *                   whose first word receives the status of cu_seqlens.
 * Errors: KDA_ERR_NULL_POINTER, KDA_ERR_INVALID_SHAPE (sizes, strides < C, channel
 * counts, width, B * T >= 2^31), KDA_ERR_INVALID_ARG (dtype, fn),
 * KDA_ERR_MISALIGNED, KDA_ERR_WORKSPACE_TOO_SMALL, KDA_ERR_UNSUPPORTED_DEVICE,
 * KDA_ERR_CUDA.
 */
KDA_API kda_status kda_conv_fwd(const void* x, int64_t x_stride, const float* weight,
                                const float* bias, void* const* outs, const int32_t* out_channels,
                                int32_t num_outs, const void* initial_state, void* final_state,
                                const int64_t* cu_seqlens, int64_t B, int64_t T, int32_t C,
                                int32_t N, int32_t width, int32_t fn, int32_t dtype,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace of kda_conv_bwd (status word and partial sums of the weights'
 * gradients). */
KDA_API kda_status kda_conv_bwd_get_workspace_size(int64_t total_tokens, int32_t C, int32_t width,
                                                   size_t* bytes);

/* kda_conv_bwd -- the gradients of <dout, out> + <dfinal_state, final_state>.
 *   douts           num_outs buffers as outs, of type dout_dtype (kda_bwd's fp32 dq,
 *                   dk, dv fit as they are).
 *   dfinal_state    NULL (zero) or [N, width - 1, C] of the rows' type.
 *   dx              [B, T, C], written in the rows' type.
 *   dweight         fp32 [C, width];  dbias fp32 [C] or NULL;  both written.
 *   dinitial_state  NULL (not written) or fp32 [N, width - 1, C].
 *   workspace       kda_conv_bwd_get_workspace_size(B * T, C, width) bytes, 128-byte
 *                   aligned. */
KDA_API kda_status kda_conv_bwd(const void* x, int64_t x_stride, const float* weight,
                                const float* bias, const void* const* douts,
                                const int32_t* out_channels, int32_t num_outs, int32_t dout_dtype,
                                const void* initial_state, const void* dfinal_state,
                                const int64_t* cu_seqlens, void* dx, float* dweight, float* dbias,
                                float* dinitial_state, int64_t B, int64_t T, int32_t C, int32_t N,
                                int32_t width, int32_t fn, int32_t dtype, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------- scan --
 * The selective state space scan, per channel d with `state` values n:
 *     delta = softplus(dt[t][d] + dt_bias[d])
 *     h_t[d][n] = exp(-delta exp(A_log[d][n])) h_{t-1}[d][n] + delta x[t][d] B[t][g][n]
 *     y[t][d]   = sum_n C[t][g][n] h_t[d][n] + D[d] x[t][d],     out = y silu(z)
 * with g = d / (dim / groups).  D, z and dt_bias may be NULL (no term, no gate,
 * zero); h starts at the sequence's initial state.  States, their gradients and saved
 * states are 16-byte aligned (KDA_ERR_MISALIGNED).  Prompts of up to 8 tokens, single ones
 * above all, have a kernel of their own, without cu_seqlens and without saved states;
 * packed single tokens take 15 times as long.
 */
typedef struct {
  const void* x;              /* rows [B, T, dim]                                    */
  const void* dt;             /* rows [B, T, dim]: raw step sizes                    */
  const void* z;              /* NULL or rows [B, T, dim]: raw gate                  */
  const void* B;              /* rows [B, T, groups * state]                         */
  const void* C;              /* rows [B, T, groups * state]                         */
  int64_t x_stride, dt_stride, z_stride, B_stride, C_stride;
  const float* A_log;         /* fp32 [dim, state]                                   */
  const float* D;             /* NULL or fp32 [dim]                                  */
  const float* dt_bias;       /* NULL or fp32 [dim]                                  */
  const void* initial_state;  /* NULL (zero) or [N, dim, state] in state_dtype       */
  const int64_t* cu_seqlens;
  int64_t batch, T;           /* batch: B                                            */
  int32_t N;                  /* sequences (taken as batch without cu_seqlens)       */
  int32_t dim, state, groups; /* state: 8, 16, 32 or 64; groups divides dim          */
  int32_t dtype;              /* kda_row_dtype of x, dt, z, B, C, out and gradients  */
  int32_t state_dtype;        /* kda_state_dtype of the initial and final states     */
} kda_scan_problem;

/* Bytes of the buffer of saved states that kda_scan_fwd writes for kda_scan_bwd: fp32
 * [slots][dim][state], the state before token KDA_SCAN_CHUNK * c of sequence n in slot
 * floor(bos_n / KDA_SCAN_CHUNK) + n + c; slots = total_tokens / KDA_SCAN_CHUNK + N + 1. */
KDA_API kda_status kda_scan_get_states_size(int64_t total_tokens, int32_t N, int32_t dim,
                                            int32_t state, size_t* bytes);
/* Bytes of workspace of kda_scan_fwd (status word, segment states of a split scan) and of
 * kda_scan_bwd (partial sums, carried gradients and, unless the caller has them, saved
 * states) for a problem; only its sizes are read, and whether cu_seqlens is NULL. */
KDA_API kda_status kda_scan_get_workspace_size(const kda_scan_problem* p, size_t* bytes);
KDA_API kda_status kda_scan_bwd_get_workspace_size(const kda_scan_problem* p, int32_t have_states,
                                                   size_t* bytes);

/* kda_scan_fwd -- out [B, T, dim] and (unless NULL) final_state [N, dim, state],
 * written; final_state may be initial_state itself.  chunk_states: NULL, or the
 * buffer of saved states (16-byte aligned), written for kda_scan_bwd.  workspace: may be
 * NULL where kda_scan_get_workspace_size is KDA_STATUS_BYTES. */
KDA_API kda_status kda_scan_fwd(const kda_scan_problem* p, void* out, void* final_state,
                                void* chunk_states, size_t chunk_states_bytes, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream);

/* kda_scan_bwd -- the gradients of <dout, out> + <dfinal_state, final_state> for the
 * forward call of the same problem.  chunk_states: NULL (recomputed), or what that
 * call saved.  dx, ddt, dz, dout: [B, T, dim]; dB, dC: [B, T, groups, state]; all in the
 * rows' type.  dA_log [dim, state], dD, ddt_bias [dim], dinitial_state [N, dim, state]:
 * fp32; dz, dD, ddt_bias and dinitial_state may be NULL (not written; dz and dD only
 * where the problem has z and D). */
KDA_API kda_status kda_scan_bwd(const kda_scan_problem* p, const void* dout,
                                const void* dfinal_state, const void* chunk_states,
                                size_t chunk_states_bytes, void* dx, void* ddt, void* dz, void* dB,
                                void* dC, float* dA_log, float* dD, float* ddt_bias,
                                float* dinitial_state, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream);

/* ------------------------------------------------------------------ norms --
 * unit(h) = h / sqrt(mean(h^2) + eps) over the last axis of dim values.
 * The scale of a residual branch, s: res_scale[dim] (fp32) where res_scale is given,
 * else the number res_scale_value.
 *
 * kda_prenorm_fwd -- before a block:
 *     residual_out = residual + s * x          out = unit(residual_out) * weight
 * (out from the sum before it is rounded to stream_dtype).
 *   x, out          rows [rows, dim] of type dtype.
 *   residual        NULL (zero) or rows of type stream_dtype (dtype or fp32).
 *   residual_out    NULL (not written) or rows of type stream_dtype; it may be residual.
 *   weight          fp32 [dim].
 *   dim             1 .. KDA_NORM_MAX_DIM.        eps  finite, >= 0.
 */
KDA_API kda_status kda_prenorm_fwd(const void* x, const void* residual, const float* weight,
                                   const float* res_scale, float res_scale_value, float eps,
                                   void* out, void* residual_out, int64_t rows, int32_t dim,
                                   int32_t dtype, int32_t stream_dtype, cudaStream_t stream);

/* Bytes of workspace of kda_prenorm_bwd and kda_postnorm_bwd (partial sums). */
KDA_API kda_status kda_norm_bwd_get_workspace_size(int64_t rows, int32_t dim, size_t* bytes);

/* kda_prenorm_bwd -- given dout, dresidual_out (NULL: zero) and the forward's
 * residual_out as `h`:
 *     dresidual = dresidual_out + (gradient of the norm),   dx = s * dresidual
 *   x               needed for dres_scale only.
 *   dx              NULL (not written; with s = 1 it equals dresidual) or rows of dtype.
 *   dresidual       NULL (not written) or rows of stream_dtype.
 *   dweight         fp32 [dim];  dres_scale NULL or fp32 [dim] (sum of dresidual * x).
 */
KDA_API kda_status kda_prenorm_bwd(const void* dout, const void* dresidual_out, const void* h,
                                   const float* weight, const void* x, const float* res_scale,
                                   float res_scale_value, float eps, void* dx, void* dresidual,
                                   float* dweight, float* dres_scale, int64_t rows, int32_t dim,
                                   int32_t dtype, int32_t stream_dtype, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/* kda_postnorm_fwd -- after a block (per head with dim the head's size):
 *     out = residual + s * (unit(x) * weight * fn(gate))
 *   x, out          rows [rows, dim] of type dtype; out may be x.
 *   gate            NULL (no gate) or rows of type dtype: row r lies at
 *                   (r / heads) * gate_stride + (r % heads) * dim.
 *   residual        NULL (zero) or rows of type dtype.
 *   fn              KDA_FN_SILU or KDA_FN_SIGMOID.
 */
KDA_API kda_status kda_postnorm_fwd(const void* x, const float* weight, const void* gate,
                                    int64_t gate_stride, int32_t heads, const void* residual,
                                    const float* res_scale, float res_scale_value, float eps,
                                    int32_t fn, void* out, int64_t rows, int32_t dim,
                                    int32_t dtype, cudaStream_t stream);

/* kda_postnorm_bwd -- the gradients of x, gate, weight and res_scale (the residual's is
 * dout).  dgate: NULL or contiguous rows; dres_scale: NULL or fp32 [dim]. */
KDA_API kda_status kda_postnorm_bwd(const void* dout, const void* x, const float* weight,
                                    const void* gate, int64_t gate_stride, int32_t heads,
                                    const float* res_scale, float res_scale_value, float eps,
                                    int32_t fn, void* dx, void* dgate, float* dweight,
                                    float* dres_scale, int64_t rows, int32_t dim, int32_t dtype,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LAYER_H_ */
