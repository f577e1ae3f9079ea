// Host-side launchers of the operators over sequences.  They assume
// validated arguments (seed_sequence_api.cpp checks everything first) and
// only enqueue work.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace seed {

constexpr int kScanChunk = 64;   // tokens of one chunk

// Parts of the recurrence's workspace, in bytes from its start; the unit of
// a part is one (slot, head), or one (token, head) for the shared keys'
// gradients.
struct ScanLayout {
  size_t n_pack;     // N (I + L beta)^-1 L, fragments of three bf16 terms
  size_t nt_pack;    // N^T
  size_t m_pack;     // M (forward) or M^T (backward)
  size_t vec;        // P, F (scalar gates) and beta, 64 floats each, 256 a unit
  size_t p, f;       // P, F of KDA, d_k floats a token
  size_t state;      // S before each chunk (backward)
  size_t grad;       // H behind each chunk (backward)
  size_t e, y;       // E, Y: d_v floats a token (backward, delta rules)
  size_t dq, dk;     // per-head gradients of keys and queries (backward: KDA, shared heads)
  size_t tp, tf;     // gradients of P and F (backward, KDA)
  size_t slow;       // 1 where a chunk's gradients go pair by pair (backward, KDA): one int
  // a long axis in segments of `seg` chunks (0: whole sequences), for each
  // (segment, head): the state a segment leaves behind zero (or the gradient
  // it passes back from zero), how it carries a state through (a matrix;
  // Mamba-2: a factor), and the state at its start (gradient at its end)
  int seg, segs;
  size_t carry, trans, start;
  size_t bytes;
};

struct ScanArgs {
  int rule;
  bool bf16;
  int n_seq, heads, key_heads, d_k, d_v, tokens;
  const int* cu;               // [n_seq + 1] or NULL: n_seq equal lengths
  const void *q, *k, *v;
  const float *g, *beta;
  const float* S0;             // or NULL: zero
  // forward
  void* o;
  float* S;
  // backward
  const void* dO;
  const float* dS;             // or NULL: zero
  void *dq, *dk, *dv;
  float *dg, *dbeta;
  float* dS0;                  // or NULL
  char* ws;
  ScanLayout at;
  int slots;                   // tokens / 64 + n_seq
};

ScanLayout scan_layout(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v, int tokens,
                       bool backward);

hipError_t launch_scan(const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t stream);

// Phases of the recurrence (seed_scan_*.hip).
hipError_t launch_scan_prep(const ScanArgs& a, bool backward, hipStream_t stream);
// From chunk to chunk: what = 0 forward, 1 forward for the backward pass
// (keeps S and E, writes no read-outs), 2 backward; in segments also 3 what
// each carries, 4 what each passes back.  chain: bf16 inputs and
// scalar gates; wide: the others.
hipError_t launch_scan_chain(const ScanArgs& a, int what, hipStream_t stream);
hipError_t launch_scan_wide(const ScanArgs& a, int what, hipStream_t stream);
// The starts of all segments from their carries (seed_scan_join.hip).
hipError_t launch_scan_join(const ScanArgs& a, bool backward, hipStream_t stream);
hipError_t launch_scan_grads(const ScanArgs& a, hipStream_t stream);

enum NormAct { kActNone = 0, kActSilu = 1, kActSigmoid = 2 };

struct NormArgs {
  long long rows;
  int groups, d;
  bool x_bf16, io_bf16;
  const void *x, *gate;
  const float *weight, *bias;   // [weight_groups][d] or NULL
  int weight_groups;
  float eps;
  bool centered, gate_first;
  int act;
  void* y;
  // backward
  const void* dy;
  void *dx, *dgate;
  float *dweight, *dbias;
  float* ws;
  int parts;                    // partial sums of dweight and dbias
};

hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream);
hipError_t launch_group_norm_backward(const NormArgs& a, hipStream_t stream);
// Partial sums the backward pass keeps per weight, for `rows` rows.
int group_norm_parts(long long rows, int groups, int d, int weight_groups);

}  // namespace seed
