// Host-side launchers of the operators on channels.  They assume validated
// arguments (seed_channels_api.cpp checks everything first) and only enqueue
// work.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace seed {

// An array over tokens: row r starts r * stride values behind p.
struct Rows {
  const void* p;
  long long stride;
};
struct OutRows {
  void* p;
  long long stride;
};

struct ConvArgs {
  int n_seq, channels, width, tokens;
  const int* cu;              // [n_seq + 1] or NULL: n_seq equal lengths
  bool bf16, silu;
  bool vectors;               // every row is one of whole aligned 16-byte vectors
  Rows x;
  const float *weight, *bias; // bias or NULL
  const void* S0;             // or NULL: zero
  // forward
  OutRows y;
  void* S;                    // or NULL
  // backward
  Rows dy;
  const void* dS;             // or NULL: zero
  OutRows dx;
  float *dweight, *dbias;     // each or NULL
  void* dS0;                  // or NULL
  float* ws;
};

hipError_t launch_short_conv(const ConvArgs& a, hipStream_t stream);
hipError_t launch_short_conv_backward(const ConvArgs& a, hipStream_t stream);
hipError_t launch_short_conv_step(const ConvArgs& a, hipStream_t stream);
// Partial sums of the weights' gradients that the backward pass keeps at most,
// each width + 1 floats a channel, for either form of its rows.
int short_conv_parts(int n_seq, int channels, int tokens);
// Whether the grids for these sizes can be launched.
bool short_conv_fits(int n_seq, int channels, int tokens);

// Parts of the scan's workspace, in bytes from its start.  A workgroup's four
// waves share a block of 64 channels, `quarter` states of each a wave; a
// channel's states are padded to 4 quarters.
struct SelectLayout {
  int quarter;      // 2, 4, 8 or 16
  int blocks;       // blocks of 64 channels of a group
  int set, sets;    // blocks that a workgroup takes one after the other, and how many such sets (backward)
  int shift;        // log2 of a segment's tokens; -1: whole sequences (forward)
  int slots;        // segments: tokens / 2^shift + n_seq
  int parts;        // workgroups over the segments (backward)
  size_t rows;      // [token][group][wave]: B and C of its states in fp32
  size_t carry;     // [slot][state][channel]: what a segment makes of zero, then its first state
  size_t back;      // the same for the gradient: what it passes back from zero, then that at its end
  size_t gone;      // [slot][channel]: sum of the scaled steps
  size_t overflow;  // [slot][block of channels][wave]: whether states grew beyond fp32 (backward)
  size_t kept;      // [8 tokens][state][channel]: what a segment makes of zero before them (backward)
  size_t before;    // [8 tokens][channel]: sum of the scaled steps before them
  size_t sums;      // [set][token][group][wave]: parts of dB and dC
  size_t weights;   // [part][state, dD, ddt_bias][channel]
  size_t bytes;
};

struct SelectArgs {
  int n_seq, channels, groups, d_state, tokens;
  const int* cu;
  bool bf16, softplus;
  Rows x, dt, B, C, z;        // z.p may be NULL
  const float *A, *D, *dt_bias, *S0;   // D, dt_bias, S0 may be NULL
  OutRows y;
  float* S;
  // backward
  Rows dy;
  const float* dS;            // or NULL: zero
  OutRows dx, ddt, dB, dC, dz;
  float *dA, *dD, *ddt_bias, *dS0;     // dD, ddt_bias, dS0 may be NULL
  char* ws;
  SelectLayout at;
};

SelectLayout select_layout(int n_seq, int channels, int groups, int d_state, int tokens, bool backward);
bool select_fits(int n_seq, int channels, int groups, int d_state, int tokens);
hipError_t launch_select(const SelectArgs& a, hipStream_t stream);
hipError_t launch_select_backward(const SelectArgs& a, hipStream_t stream);
// n_seq: the batch; x, dt, B, C, z, y one row each.
hipError_t launch_select_step(const SelectArgs& a, hipStream_t stream);

}  // namespace seed
