/*
 * seed_channels.h -- operators on channels, beside the heads' operators of
 * seed_sequence.h: the short causal convolution in front of a recurrence, and
 * the selective state space scan (a state of its own for every channel, with
 * steps, inputs and read-outs that come with the token).  Each runs over whole
 * sequences, backward, and for single tokens.
 *
 * The conventions of seed_sequence.h hold: device pointers owned by the
 * caller, `stream` a hipStream_t, arguments validated on the host before any
 * HIP call, a seed_status back, seed_last_error() for the reason, no result
 * that depends on the order of atomics, nothing kept between calls.
 *
 * Arrays over tokens have rows: row r of `x` starts x_stride values behind row
 * r - 1 and holds its values one behind the other, so that a slice of a wider
 * array (a projection's rows) can be given as it is.  Strides are at least the
 * row's length; such arrays have to be aligned to their own type only (16-byte
 * rows of a multiple of 8 channels are the fast ones).  Everything else is
 * dense and row-major with a 16-byte aligned base.
 *
 * cu_seqlens (int [n_seq + 1], device): sequence s is rows cu_seqlens[s] ..
 * cu_seqlens[s + 1] - 1, 0 <= cu_seqlens[s] <= cu_seqlens[s + 1] <= tokens.
 * NULL: n_seq sequences of tokens / n_seq rows each.  Sequences may be empty.
 * Rows of outputs outside every sequence are left as they were.  Offsets that
 * break the order give wrong results but no access outside the arrays.
 * Outputs and workspaces must not overlap inputs (cu_seqlens is one) or each
 * other, but where it is said.
 */
#ifndef SEED_CHANNELS_H
#define SEED_CHANNELS_H

#include "seed_sequence.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * seed_short_conv -- y_t = act(bias + sum_j weight[j] x_{t - (width - 1) + j})
 * for every channel by itself, j = 0 .. width - 1, within each sequence.
 *
 *   x, y     [tokens] rows of `channels`, fp32 or bf16 (io_dtype)
 *   weight   float [channels][width], width 2, 3 or 4
 *   bias     float [channels] or NULL
 *   S0, S    [n_seq][width - 1][channels] of io_dtype: the inputs of the
 *            last width - 1 tokens, the oldest first.  S0: those before each
 *            sequence (NULL: zero).  S: those behind it; may be NULL, may be
 *            S0.  An empty sequence's S is its S0.
 *   activation  SEED_ACT_NONE or SEED_ACT_SILU
 *
 * Sums are fp32; y is rounded once.  A NaN or infinity reaches the width
 * tokens that it is a tap of.  channels <= 2^20.
 */
seed_status seed_short_conv(int n_seq, int channels, int width, int tokens, const int *cu_seqlens,
                            const void *x, long long x_stride, int io_dtype, const float *weight,
                            const float *bias, const void *S0, int activation, void *y,
                            long long y_stride, void *S, void *stream);

/*
 * seed_short_conv_backward -- gradients of seed_short_conv's inputs from dy
 * and dS (that of S; NULL: zero): dx (io_dtype), dweight and dbias (fp32,
 * summed in an order fixed by the sizes; each may be NULL), dS0 (io_dtype, may
 * be NULL).  The pre-activations are computed again from x.
 */
seed_status seed_short_conv_backward(int n_seq, int channels, int width, int tokens,
                                     const int *cu_seqlens, const void *x, long long x_stride,
                                     int io_dtype, const float *weight, const float *bias,
                                     const void *S0, int activation, const void *dy,
                                     long long dy_stride, const void *dS, void *dx,
                                     long long dx_stride, float *dweight, float *dbias, void *dS0,
                                     void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace for seed_short_conv_backward with dweight or dbias;
 * (size_t)-1 for sizes it rejects. */
size_t seed_short_conv_workspace_bytes(int n_seq, int channels, int width, int tokens);

/*
 * seed_short_conv_step -- one token of `batch` sequences: row b of x continues
 * the inputs in S0[b], y is its convolution, S[b] the inputs behind it.
 * S0, S [batch][width - 1][channels] of io_dtype; S may be S0 (the step in
 * place).  y may be x where their strides are equal.
 */
seed_status seed_short_conv_step(int batch, int channels, int width, const void *x,
                                 long long x_stride, int io_dtype, const float *weight,
                                 const float *bias, const void *S0, int activation, void *y,
                                 long long y_stride, void *S, void *stream);

/*
 * seed_selective_scan -- for every channel c, in group g = c / (channels /
 * groups), with states n = 0 .. d_state - 1:
 *   delta_t = softplus(dt_t + dt_bias)  (dt_t + dt_bias unless `softplus`)
 *   h_t[n]  = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[g][n]
 *   y_t     = (sum_n C_t[g][n] h_t[n] + D x_t) silu(z_t)
 * from S0 (NULL: zero), leaving the last states in S.
 *
 *   x, dt, z, y  [tokens] rows of `channels`, fp32 or bf16 (io_dtype); z may
 *                be NULL (no gate)
 *   B, C         [tokens] rows of [groups][d_state], the same type
 *   A            float [channels][d_state], the rates (negative for decay)
 *   D, dt_bias   float [channels], each may be NULL (0)
 *   S0, S        float [n_seq][channels][d_state]; S may be S0
 *   softplus     softplus(v) = log(1 + exp(v)), or 0: v itself
 *
 * Steps, states and sums are fp32, y is rounded once.  Where a batch has few
 * sequences, they are run in segments that are joined through the workspace; a
 * segment's decay is exp(A sum(delta)), off by at most |A sum(delta)| 2^-17 of
 * its value.  The choice goes by the number of sequences and their mean length:
 * one that is much longer than the many others of its batch is run from end to
 * end (0.18 us a token), and is faster in a call of its own.
 *
 * An exponential is off by about (1 + |delta A|) 2^-23 of its value; decays below
 * 2^-126, also products of them, are zero.  States may grow (A delta > 0), by any
 * factor over a segment: where each step's exponential is finite, and the states
 * (backwards, the gradients) are with the magnitudes of their terms, so are the
 * results.  A rate of -infinity is taken as the lowest fp32 number: its states
 * keep nothing over a step (above 2^-120) but are left by a step of zero;
 * gradients the same.  A NaN or infinity of a token's x, dt or z stays in its
 * channel (of B or C: in its group) and in its sequence; an infinity may come out
 * as NaN.
 * channels a multiple of groups and <= 2^20, d_state 1 .. 64.
 */
seed_status seed_selective_scan(int n_seq, int channels, int groups, int d_state, int tokens,
                                const int *cu_seqlens, const void *x, long long x_stride,
                                const void *dt, long long dt_stride, const float *A, const void *B,
                                long long B_stride, const void *C, long long C_stride,
                                int io_dtype, const float *D, const void *z, long long z_stride,
                                const float *dt_bias, int softplus, const float *S0, void *y,
                                long long y_stride, float *S, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * seed_selective_scan_backward -- gradients of seed_selective_scan's inputs
 * from dy and dS (that of S; NULL: zero): dx, ddt, dB, dC and dz (io_dtype;
 * dz given exactly if z is), dA and, where given, dD, ddt_bias and dS0
 * (fp32).  dD and ddt_bias may be asked for where D or dt_bias is NULL.  dB
 * and dC are the sums over their group's channels, dA, dD and ddt_bias over
 * all tokens, in fp32 in an order fixed by the sizes; each gradient is
 * rounded once.  Nothing from seed_selective_scan is needed: the states are
 * run again.  dS0 may be dS.
 */
seed_status seed_selective_scan_backward(
    int n_seq, int channels, int groups, int d_state, int tokens, const int *cu_seqlens,
    const void *x, long long x_stride, const void *dt, long long dt_stride, const float *A,
    const void *B, long long B_stride, const void *C, long long C_stride, int io_dtype,
    const float *D, const void *z, long long z_stride, const float *dt_bias, int softplus,
    const float *S0, const void *dy, long long dy_stride, const float *dS, void *dx,
    long long dx_stride, void *ddt, long long ddt_stride, float *dA, void *dB, long long dB_stride,
    void *dC, long long dC_stride, float *dD, void *dz, long long dz_stride, float *ddt_bias,
    float *dS0, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace for seed_selective_scan (backward = 0) or
 * seed_selective_scan_backward (backward = 1); (size_t)-1 for sizes they
 * reject. */
size_t seed_selective_scan_workspace_bytes(int n_seq, int channels, int groups, int d_state,
                                           int tokens, int backward);

/*
 * seed_selective_step -- one token of `batch` sequences: seed_selective_scan
 * of one row each, from S0 to S (float [batch][channels][d_state], S may be
 * S0: the step in place).  y may be x, dt or z where their strides are equal.
 */
seed_status seed_selective_step(int batch, int channels, int groups, int d_state, const void *x,
                                long long x_stride, const void *dt, long long dt_stride,
                                const float *A, const void *B, long long B_stride, const void *C,
                                long long C_stride, int io_dtype, const float *D, const void *z,
                                long long z_stride, const float *dt_bias, int softplus,
                                const float *S0, void *y, long long y_stride, float *S,
                                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SEED_CHANNELS_H */
