// The selective state space scan: what its kernels share.  For one channel of
// a group, states n:
//   v_t = dt_t + dt_bias,  delta_t = softplus(v_t) or v_t,  a_t = exp(delta_t A)
//   h_t = a_t h_{t-1} + delta_t x_t B_t,   s_t = C_t.h_t + D x_t,   y_t = s_t silu(z_t)
// and backwards, with G_t the gradient of h_t and ds_t = dy_t silu(z_t):
//   G_t = ds_t C_t + a_{t+1} G_{t+1} (+ dS behind the last token)
//   dC_t = sum over channels ds_t h_t,  dB_t = sum over channels G_t delta_t x_t
//   du_t = G_t.B_t,  r_t = G_t a_t h_{t-1},  dA = sum over t delta_t r_t
//   ddelta_t = x_t du_t + A.r_t,  dx_t = delta_t du_t + D ds_t
//   ddt_t = ddelta_t softplus'(v_t),  dz_t = dy_t s_t silu'(z_t).
//
// A lane is a channel and keeps 16 of its states in registers, so that the
// sums over states stay in the lane, and B and C of a token, the same for a
// wave's channels, are scalar operands: they are read through the scalar cache
// from fp32 rows, padded to whole sixteens (prepare_kernel).  For d_state
// above 16, 2 or 4 waves of a workgroup share a block of channels.
#pragma once

#include "seed_channels.h"

namespace seed {
namespace channels {

constexpr int kStates = 16;     // a lane's
constexpr int kWaves = 4;       // of a workgroup
constexpr int kTile = 8;        // tokens whose inputs are on their way together
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

typedef const __attribute__((address_space(4))) float* ScalarRow;   // read by scalar loads

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|), and its slope
// 1 / (1 + exp(-v)).  log(1 + e) = 2 atanh(e / (2 + e)): with s = e / (2 + e)
// at most 1/3, atanh(s) / s is a polynomial in s^2, here of degree 4 (fitted
// on Chebyshev points; 4e-9 of the value), so that small values keep their
// relative accuracy.
struct Step {
  float v;
  __device__ __forceinline__ float of(bool softplus) const {
    if (!softplus) return v;
    const float e = exp2_fast(fabsf(v) * -kLog2e);
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
    float p = 0.14087337f;
    p = p * q + 0.139807165f;
    p = p * q + 0.20012425f;
    p = p * q + 0.333331585f;
    p = p * q + 1.f;
    return fmaxf(v, 0.f) + 2.f * s * p;
  }
  __device__ __forceinline__ float slope(bool softplus) const {
    return softplus ? sigmoid(v) : 1.f;
  }
};

// Which channels and states a wave of a workgroup has.
struct Mine {
  int group, c, sb;     // c: clamped to the group's channels
  int block;            // the workgroup's among the group's
  bool live;
};
template <int SB>
__device__ __forceinline__ Mine mine(const SelectArgs& a, int block) {
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), each = a.channels / a.groups;
  Mine m;
  m.group = block / a.at.blocks;
  m.block = block - m.group * a.at.blocks;
  m.sb = wave % SB;
  const int in = (m.block * (kWaves / SB) + wave / SB) * 64 + (int)__lane_id();
  m.live = in < each;
  m.c = m.group * each + (in < each ? in : each - 1);
  return m;
}

// Index of a state of channel c among the user's [.][channels][d_state].
__device__ __forceinline__ size_t state_at(const SelectArgs& a, int of, int c) {
  return ((size_t)of * a.channels + c) * a.d_state;
}
// ... and among the workspace's [slot][16 waves states][channels].
template <int SB>
__device__ __forceinline__ size_t carry_at(const SelectArgs& a, int slot, int n, int c) {
  return ((size_t)slot * (SB * kStates) + n) * a.channels + c;
}

// A in powers of two: exp(delta A) = 2^(delta A log2 e).
template <int SB>
__device__ __forceinline__ void load_rates(const SelectArgs& a, const Mine& m, float (&A)[kStates]) {
#pragma unroll
  for (int i = 0; i < kStates; ++i) {
    const int n = m.sb * kStates + i;
    A[i] = n < a.d_state ? a.A[(size_t)m.c * a.d_state + n] * kLog2e : 0.f;
  }
}

// B (and, 16 SB floats on, C) of a token for a wave's states.
template <int SB>
__device__ __forceinline__ ScalarRow row_bc(const SelectArgs& a, const Mine& m, int t) {
  return (ScalarRow)(uintptr_t)(a.ws + a.at.rows) +
         ((size_t)t * a.groups + m.group) * (2 * SB * kStates) + m.sb * kStates;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const Rows& r, long long t) {
  return static_cast<const T*>(r.p) + t * r.stride;
}
template <typename T>
__device__ __forceinline__ T* row_of(const OutRows& r, long long t) {
  return static_cast<T*>(r.p) + t * r.stride;
}

}  // namespace channels

hipError_t launch_select_prepare(const SelectArgs& a, hipStream_t stream);
// First states (and the gradients at the ends) of the segments from what each
// carries; S and dS0 of whole sequences.
hipError_t launch_select_join(const SelectArgs& a, bool backward, hipStream_t stream);

}  // namespace seed
