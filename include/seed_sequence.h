/*
 * seed_sequence.h -- operators over whole sequences, beside the single-token
 * steps of seed.h: the gated linear recurrence (prefill) and its backward
 * pass, and the group norm with a gate that follows the read-outs, forward
 * and backward.
 *
 * The conventions of seed.h hold: device pointers owned by the caller, dense
 * row-major arrays, base pointers 16-byte aligned, `stream` a hipStream_t,
 * arguments validated on the host before any HIP call, a seed_status back,
 * seed_last_error() for the reason.  The library keeps nothing between
 * calls; a workspace is the caller's, may be shared by calls that a stream
 * orders one after the other, and holds nothing afterwards.  No result
 * depends on the order of atomics: the same call gives the same bits.
 */
#ifndef SEED_SEQUENCE_H
#define SEED_SEQUENCE_H

#include "seed.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * seed_scan -- run the recurrence of a rule (seed_rule) over sequences:
 *   S_t = the head's update of S_{t-1} by token t,   o_t = S_t^T q_t
 * for every token of every sequence and head, starting from S0 (NULL: zero)
 * and leaving the last state in S.  It is dense_decode_step for each token,
 * computed 64 tokens at a time; S feeds seed_state_from_dense.
 *
 *   q, k   [tokens][key_heads][d_k]   fp32 or bf16 (in_dtype); head h reads
 *                                     key head h / (heads / key_heads)
 *   v, o   [tokens][heads][d_v]       the same type
 *   g      float [tokens][heads]      decay (Gated DeltaNet, Mamba-2)
 *          float [tokens][heads][d_k] decay per key channel (KDA)
 *   beta   float [tokens][heads]      write strength (NULL for Mamba-2)
 *   S0, S  float [n_seq][heads][d_k][d_v]   may be the same array
 *   cu_seqlens  int [n_seq + 1], device: sequence s is tokens cu_seqlens[s]
 *          .. cu_seqlens[s + 1] - 1 of the arrays, 0 <= cu_seqlens[s] <=
 *          cu_seqlens[s + 1] <= tokens.  NULL: n_seq sequences of tokens /
 *          n_seq tokens each.  Sequences may be empty (S = S0); rows of o
 *          outside every sequence are left as they were, and inputs there
 *          are not read.  Offsets that break the order give wrong results
 *          but no access outside the arrays.
 *
 * Gates may be 0.  A head's scalar gates enter as products only; gates per
 * key channel as quotients of products where those of 64 tokens stay within
 * 2^-60 .. 2^60, as products otherwise.  Logarithms are never taken.
 * Sums and states are fp32; the products run on the matrix cores with an fp32
 * operand as three bf16 terms (2^-27 of it is left out), whatever the inputs'
 * type: the last state of 512 tokens is within 1e-6 of its norm, also with
 * gates of 1 or keys that point one way.  A NaN or infinity of a token
 * reaches its sequence's state and read-outs from the first token of its 64
 * on, and no other sequence.  A finite float32 above 3.39e38, where bf16 ends,
 * counts as one.
 * Outputs and the workspace must not overlap inputs (cu_seqlens is one) or
 * each other (S may be S0).
 * 1 <= key_heads <= heads, heads a multiple of key_heads, heads <= 65535;
 * d_k, d_v as in seed.h.
 */
seed_status seed_scan(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v, int tokens,
                      const int *cu_seqlens, const void *q, const void *k, const void *v,
                      int in_dtype, const float *g, const float *beta, const float *S0, void *o,
                      float *S, void *workspace, size_t workspace_bytes, void *stream);

/*
 * seed_scan_backward -- the gradients of seed_scan's inputs, given dO, the
 * gradient of o (in_dtype), and dS, that of the last states (NULL: zero).
 * dq, dk, dv have the inputs' shapes and type, dg and dbeta are fp32 (dbeta
 * NULL for Mamba-2), dS0 may be NULL.  dq and dk of a shared key head are
 * the sums over its heads, in fp32, rounded once.  Nothing from seed_scan is
 * needed: the states are run again.  Rows outside every sequence are left as
 * they were.  Gradients and the workspace must not overlap inputs or each
 * other (dS0 may be dS).
 */
seed_status seed_scan_backward(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v,
                               int tokens, const int *cu_seqlens, const void *q, const void *k,
                               const void *v, int in_dtype, const float *g, const float *beta,
                               const float *S0, const void *dO, const float *dS, void *dq,
                               void *dk, void *dv, float *dg, float *dbeta, float *dS0,
                               void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace for seed_scan (backward = 0) or seed_scan_backward
 * (backward = 1); (size_t)-1 for arguments they reject. */
size_t seed_scan_workspace_bytes(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v,
                                 int tokens, int backward);

typedef enum {
  SEED_ACT_NONE = 0,
  SEED_ACT_SILU = 1,    /* x / (1 + exp(-x)) */
  SEED_ACT_SIGMOID = 2  /* 1 / (1 + exp(-x)) */
} seed_activation;

/*
 * seed_group_norm -- normalise each group of d channels of each row, then
 * scale, shift and gate:
 *   h   = x act(gate) if gate_first, else x
 *   hat = (h - mean) / sqrt(mean((h - mean)^2) + eps)   (mean taken as 0
 *         unless `centered`)
 *   n   = hat weight + bias
 *   y   = n act(gate), n if gate_first, act(n) if gate is NULL
 *
 *   x       [rows][groups][d]  fp32 or bf16 (x_dtype)
 *   gate, y [rows][groups][d]  fp32 or bf16 (io_dtype); gate may be NULL
 *   weight, bias  float [weight_groups][d], weight_groups 1 (shared by the
 *           groups) or `groups`; each may be NULL (1 and 0)
 * A head's norm behind the read-outs has groups = heads and d = d_v; the
 * norm over a layer's whole width has groups = 1.  Everything between load
 * and store is fp32.  y may be x or gate where the types are the same.
 * 1 <= d <= 8192; rows may be 0.  gate_first needs a gate.
 */
seed_status seed_group_norm(long long rows, int groups, int d, const void *x, int x_dtype,
                            const void *gate, int io_dtype, const float *weight,
                            const float *bias, int weight_groups, float eps, int centered,
                            int activation, int gate_first, void *y, void *stream);

/*
 * seed_group_norm_backward -- gradients of seed_group_norm given dy
 * (io_dtype): dx (x_dtype), dgate (io_dtype; given exactly if gate is),
 * dweight and dbias (fp32, shapes of weight and bias; each may be NULL, and
 * dweight or dbias may be asked for where weight or bias is NULL).  The
 * statistics are computed again from x.  dweight and dbias are summed in
 * fp32 over blocks of rows, in an order fixed by the sizes; with rows = 0
 * they are zero.  dx may be x, dgate may be gate or dy, dx may be dy (where
 * the types are the same).  workspace: seed_group_norm_workspace_bytes().
 */
seed_status seed_group_norm_backward(long long rows, int groups, int d, const void *dy,
                                     const void *x, int x_dtype, const void *gate, int io_dtype,
                                     const float *weight, const float *bias, int weight_groups,
                                     float eps, int centered, int activation, int gate_first,
                                     void *dx, void *dgate, float *dweight, float *dbias,
                                     void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace for seed_group_norm_backward; (size_t)-1 for sizes it
 * rejects. */
size_t seed_group_norm_workspace_bytes(long long rows, int groups, int d, int weight_groups);

#ifdef __cplusplus
}
#endif

#endif /* SEED_SEQUENCE_H */
