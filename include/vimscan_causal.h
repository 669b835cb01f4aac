/*
 * vimscan_causal.h -- C ABI of libvimscan.so's causal operators: the S6 recurrence and its
 * short convolution in one direction, with the state handed in and out, for models that
 * read a sequence once from its start ("Vision Mamba Guide", sections "The Selective State
 * Space (S6) Mechanism" and "2. The Bidirectional Mamba Block", the forward pathway alone);
 * their derivatives; and clipping by the common norm of many gradients.
 *
 * The conventions of vimscan.h hold, and:
 *   - Activations are given by rows (vim_rows), so that a half of one projection's
 *     output or a few of its columns can be passed as they lie.  Any channel count is
 *     taken; rows less than 2^29 elements apart.  Offsets are 64-bit.  Rows that start on
 *     16-byte boundaries and hold whole 16-byte vectors move faster (convolution).
 *   - Sequences (vim_sequences) are the batch rows, or ranges of one packed row.
 *   - Tables on the device (offsets, slots) are not seen by the host checks.  The kernels
 *     bound them: no value leads to an access outside the tensors.
 *   - Inputs and outputs are aligned to their elements unless stated otherwise.
 *   - An output must not overlap another tensor of the call except where it is said that it
 *     may be an input.  Overlapping rows are refused where their strides are the same or
 *     they start at the same address (VIM_ERR_INVALID_ARG); other overlaps are not seen.
 */
#ifndef VIMSCAN_CAUSAL_H
#define VIMSCAN_CAUSAL_H

#include "vimscan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of channels: element (b, t, c) is data[b * batch_stride + t * row_stride + c],
 * strides in elements. */
typedef struct {
    const void *data;
    int64_t batch_stride, row_stride;
} vim_rows;

/*
 * The sequences of a call and their states.
 *   cu_seqlens : NULL: one sequence per batch row, of L tokens.  Else DEVICE int32
 *                [n_seqs + 1], non-decreasing: sequence s holds tokens cu_seqlens[s] ..
 *                cu_seqlens[s+1] - 1 of the single row of L packed tokens (batch = 1);
 *                empty sequences are allowed.  Tokens before the first and after the last
 *                sequence belong to none: outputs there are left as they were.
 *   state      : initial states, one row of n_slots rows per sequence, or NULL (zeros).
 *   state_out  : receives the final states, or NULL.  May be `state` itself (in place);
 *                otherwise it must not overlap it, and rows of no sequence stay untouched.
 *   slots      : DEVICE int32 [n_seqs], the state row of each sequence, or NULL (sequence s
 *                has row s).  A value outside 0 .. n_slots - 1 marks a padding entry: that
 *                sequence is skipped, its outputs are left as they were.  Two sequences
 *                must not name the same row; if they do, that row ends as one of them left
 *                it (in place, either may have started from the other's result).
 *   fresh      : DEVICE bytes [n_seqs], or NULL.  Non-zero: the sequence starts from zeros
 *                whatever its state row holds.
 */
typedef struct {
    const int32_t *cu_seqlens;
    int64_t n_seqs;
    const void *state;
    void *state_out;
    const int32_t *slots;
    int64_t n_slots;
    const unsigned char *fresh;
} vim_sequences;

/*
 * Causal selective scan:
 *   h_t = exp(Delta_t A) h_(t-1) + Delta_t B_t u_t,  Delta_t = softplus(delta_t + delta_bias)
 *   y_t = (C_t . h_t + D u_t) * silu(z_t)
 *   u, delta, z, y : rows of d_inner channels (dt); z.data may be NULL (no gate).  y may be
 *                    u, delta or z itself (the same rows); it must not overlap anything else.
 *   B, C           : rows of d_state (dt), shared by all channels of a token.
 *   A              : [d_inner, d_state] fp32, 16-byte aligned, meant to be <= 0, -infinity
 *                    included (of any values; with A > 0 the decays of 16 tokens together
 *                    must stay finite); D, delta_bias : [d_inner] fp32.
 *   seqs           : NULL: batch rows, no states.  States are fp32 [n_slots, d_inner,
 *                    d_state], 16-byte aligned, and finite: one that is infinite, given or
 *                    by an overflow, may become NaN where it would stay infinite token by
 *                    token.
 *   ckpt           : NULL, or fp32 causal_ckpt_bytes(batch, L, d_inner, d_state) bytes,
 *                    16-byte aligned: the state entering every 8th token of a row,
 *                    [batch, ceil(L / 8), d_inner, d_state], for causal_scan_bwd; those
 *                    of padding entries too.  Not together with initial states
 *                    (VIM_ERR_INVALID_ARG): the derivative starts every sequence from
 *                    zeros.
 * One launch, no workspace.
 */
typedef struct {
    vim_rows u, delta, z, B, C, y;
} vim_scan_io;
vim_status causal_scan(const vim_scan_io *io, const float *A, const float *D, const float *delta_bias, int batch,
                       int L, int d_inner, int d_state, vim_dtype dt, const vim_sequences *seqs, float *ckpt,
                       cudaStream_t stream);
size_t causal_ckpt_bytes(int batch, int L, int d_inner, int d_state);

/*
 * causal_scan for one token of each of `batch` sequences (seqs->n_seqs = batch, cu_seqlens
 * ignored): u, delta, z, B, C, y are rows (b, 0) of batch_stride elements each.  state is
 * required; state_out NULL means in place.
 */
vim_status causal_scan_step(const vim_scan_io *io, const float *A, const float *D, const float *delta_bias,
                            int batch, int d_inner, int d_state, vim_dtype dt, const vim_sequences *seqs,
                            cudaStream_t stream);

/*
 * Derivative of causal_scan for sequences that start from zeros and whose final states are
 * not used, for a loss with derivative `dout` with respect to y.
 *   u, delta, z, B, C, A, D, delta_bias : the forward call's inputs; dout : rows (dt).
 *   du, ddelta, dz : rows (dt), written; ddelta is with respect to the raw delta; dz.data
 *               NULL exactly when z.data is.
 *   dB, dC    : fp32 [batch, L, d_state], contiguous, written.
 *   dA [d_inner, d_state], dD [d_inner], ddelta_bias [d_inner] : fp32, written.
 *   cu_seqlens, n_seqs : as in vim_sequences (NULL: one sequence per batch row).  Rows of
 *               no sequence keep what they held in every output.  There are no slots here:
 *               a sequence that causal_scan skipped as a padding entry is differentiated
 *               like any other, so its dout is to be zero and its inputs finite (or the
 *               offsets are to leave it out).
 *   ckpt      : what causal_scan kept for the same inputs, or NULL: formed here.
 *   workspace : causal_bwd_workspace_bytes(batch, L, d_inner, d_state, ckpt != NULL) bytes,
 *               256-byte aligned.
 * Every sum is taken in a fixed order.  No token at all writes zero derivatives of the
 * parameters.
 */
typedef struct {
    vim_rows u, delta, z, B, C, dout, du, ddelta, dz;
} vim_scan_bwd_io;
vim_status causal_scan_bwd(const vim_scan_bwd_io *io, const float *A, const float *D, const float *delta_bias,
                           float *dB, float *dC, float *dA, float *dD, float *ddelta_bias, int batch, int L,
                           int d_inner, int d_state, vim_dtype dt, const int32_t *cu_seqlens, int n_seqs,
                           const float *ckpt, void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t causal_bwd_workspace_bytes(int batch, int L, int d_inner, int d_state, int has_ckpt);

/*
 * Short causal depthwise convolution, the front of the causal scan ("1D Conv -> SiLU", here
 * over the past only):
 *   pre[b,t,c] = b[c] + sum_k w[c][k] x[b, t - width + 1 + k, c],   k = 0 .. width - 1
 *   y = silu(pre) where `silu` is non-zero, else pre
 *   x, y   : rows of `channels` (dt); y must not overlap x.
 *   w      : [channels, width] fp32, width 2, 3 or 4 (the newest tap last); b : [channels]
 *            fp32 or NULL.
 *   seqs   : states are [n_slots, width - 1, channels] (dt), aligned to their elements: the
 *            last width - 1 inputs of the sequence, oldest first.
 * Sums are formed in fp32 and rounded once.
 */
typedef struct {
    vim_rows x, y;
} vim_conv_io;
vim_status causal_conv(const vim_conv_io *io, const float *w, const float *b, int batch, int L, int channels,
                       int width, int silu, vim_dtype dt, const vim_sequences *seqs, cudaStream_t stream);
/* causal_conv for one token of each of `batch` sequences, rows as in causal_scan_step; state is
 * required, state_out NULL means in place; y may be x itself. */
vim_status causal_conv_step(const vim_conv_io *io, const float *w, const float *b, int batch, int channels,
                            int width, int silu, vim_dtype dt, const vim_sequences *seqs, cudaStream_t stream);
/*
 * Derivative of causal_conv for sequences that start from zeros and whose final states are
 * not used.  dout, dx : rows (dt), dx written; dw [channels, width] and db [channels] (NULL
 * where b is, or where it is not wanted) : fp32, written.  cu_seqlens, n_seqs as in
 * causal_scan_bwd; rows of no sequence keep what dx held.  workspace :
 * causal_conv_bwd_workspace_bytes(batch, L, channels, width) bytes, 256-byte aligned.  Every
 * sum is taken in a fixed order.
 */
typedef struct {
    vim_rows x, dout, dx;
} vim_conv_bwd_io;
vim_status causal_conv_bwd(const vim_conv_bwd_io *io, const float *w, const float *b, float *dw, float *db,
                           int batch, int L, int channels, int width, int silu, vim_dtype dt,
                           const int32_t *cu_seqlens, int n_seqs, void *workspace, size_t workspace_bytes,
                           cudaStream_t stream);
size_t causal_conv_bwd_workspace_bytes(int batch, int L, int channels, int width);

/* A gradient tensor: n elements of type dtype (VIM_F32 or VIM_BF16) at data, and where its
 * clipped values go (out == data: in place). */
typedef struct {
    const void *data;
    void *out;
    int64_t n;
    int64_t dtype;
} vim_tensor;

/*
 * The common norm of `count` gradient tensors, and clipping by it (what a training step does
 * with everything the derivatives above return):
 *   norm  = sqrt(sum over all elements of g^2)         -> *norm (DEVICE, one float)
 *   out_i = g_i * min(1, max_norm / (norm + 1e-6)), rounded once to the tensor's type
 *   tensors   : HOST array; the tensors are in device memory, aligned to their elements,
 *               contiguous, empty ones allowed.  An `out` must not overlap any other tensor.
 *   max_norm  : >= 0; infinity clips nothing and, in place, writes nothing but the norm.
 *   workspace : clip_grad_norm_workspace_bytes(count) bytes, 256-byte aligned.
 * The norm and the workspace must not overlap a tensor.  A norm that is NaN or infinite (in
 * fp32) clips nothing: `out` gets the gradients as they are, and the caller sees the norm.
 * The sum is formed in fp64 in a fixed order.  Two launches for every 120 tensors.
 */
vim_status clip_grad_norm(const vim_tensor *tensors, int count, float max_norm, float *norm, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream);
size_t clip_grad_norm_workspace_bytes(int count);

#ifdef __cplusplus
}
#endif

#endif /* VIMSCAN_CAUSAL_H */
