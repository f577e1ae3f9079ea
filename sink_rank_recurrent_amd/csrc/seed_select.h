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
// A lane is a channel; the four waves of a workgroup have the same 64
// channels and a quarter of the states each, in registers.  What a token needs
// once per channel (softplus, gate, the gradients of x, dt and z) is shared
// out among the waves, two of every eight tokens each, and goes through LDS.
// B and C of a token are the same for a wave's lanes: they are scalar operands,
// read through the scalar cache from fp32 rows (prepare_kernel).
#pragma once

#include "seed_channels.h"

namespace seed {
namespace channels {

constexpr int kWaves = 4;       // of a workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 8;        // tokens that go through LDS together
constexpr int kOwn = kTile / kWaves;   // of them prepared by one wave
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

// A wave's channels and states.
struct Mine {
  int group, c, wave;   // c: clamped to the group's channels
  bool live;
};
__device__ __forceinline__ Mine mine(const SelectArgs& a, int group, int block) {
  const int each = a.channels / a.groups, in = block * 64 + (int)__lane_id();
  return {group, group * each + (in < each ? in : each - 1),
          __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), in < each};
}

// Index of a state of channel c among the user's [.][channels][d_state].
__device__ __forceinline__ size_t state_at(const SelectArgs& a, int of, int c) {
  return ((size_t)of * a.channels + c) * a.d_state;
}
// ... and among the workspace's [.][4 Q states][channels].
template <int Q>
__device__ __forceinline__ size_t carry_at(const SelectArgs& a, int of, int n, int c) {
  return ((size_t)of * (4 * Q) + n) * a.channels + c;
}

// A in powers of two: exp(delta A) = 2^(delta A log2 e).
template <int Q>
__device__ __forceinline__ void load_rates(const SelectArgs& a, const Mine& m, float (&A)[Q]) {
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int n = m.wave * Q + i;
    A[i] = n < a.d_state ? a.A[(size_t)m.c * a.d_state + n] * kLog2e : 0.f;
  }
}

// B and C of the tokens of a tile for a wave's states.  `last`: the last token
// of the sequence or segment, counted from the tile's first; tokens behind it
// take its row (their steps are zero, but a row of another sequence may hold
// an infinity).
template <int Q>
struct TileRows {
  uintptr_t base;
  uint32_t step;
  int last;
  __device__ __forceinline__ TileRows(const SelectArgs& a, const Mine& m, int t, int t1)
      : base((uintptr_t)(a.ws + a.at.rows) + (((size_t)t * a.groups + m.group) * 4 + m.wave) * (8 * Q)),
        step((uint32_t)a.groups * (32 * Q)), last(t1 - 1 - t) {}
  __device__ __forceinline__ ScalarRow operator[](int j) const {
    return (ScalarRow)(base + (uint32_t)(j < last ? j : last) * step);
  }
};
// The tile's rows in scalar registers where those suffice (Q <= 4: 64 of them,
// on their way while the steps are made); else each token's when it is used.
template <int Q>
struct Scalars {
  float v[Q <= 4 ? kTile : 1][2 * Q];
  TileRows<Q> rows;
  __device__ __forceinline__ explicit Scalars(const TileRows<Q>& r) : rows(r) {
    if constexpr (Q <= 4) {
#pragma unroll
      for (int j = 0; j < kTile; ++j)
#pragma unroll
        for (int i = 0; i < 2 * Q; ++i) v[j][i] = rows[j][i];
    }
  }
  // B and, Q floats on, C of token j
  __device__ __forceinline__ const float* of(int j) {
    if constexpr (Q <= 4) {
      return v[j];
    } else {
#pragma unroll
      for (int i = 0; i < 2 * Q; ++i) v[0][i] = rows[j][i];
      return v[0];
    }
  }
};
// Nothing is moved over this point: what a token needs, in registers or on its
// way, does not pile up with the other tokens'.
__device__ __forceinline__ void next_token() { __builtin_amdgcn_sched_barrier(0); }

// The call's arguments, read again from where the launch put them: pointers and
// strides of a dozen arrays, each used once a tile, would take the scalar
// registers that the rows of B and C need.
typedef const __attribute__((address_space(4))) SelectArgs* ArgsAgain;
__device__ __forceinline__ ArgsAgain args_again() {
  auto p = (ArgsAgain)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
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
