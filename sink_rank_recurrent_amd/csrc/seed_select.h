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
// B and C of a token are the same for a wave's lanes; they come from fp32 rows
// (prepare_kernel), a tile's through LDS.  Where they multiply a state each
// (C.h, G.B) they are scalar operands or read from LDS, the same in every lane.
// Where they make an outer product with the channels (h += B u, G += C ds) a
// matrix instruction of 4 x 4 blocks adds four states of 64 channels at once:
// 4 x 1 values of a token's row, the same in every block, times 1 x 4 channels,
// onto accumulators that lie as the states do.
//
// A state of a token costs an exponential (two issue slots of the vector unit;
// the hardware's, base 2, one unit in the last place) and at least four
// operations forward and eleven backward, against a few bytes for its channel:
// the vector unit bounds the scan, and what is not done for each state has to
// be shared or taken off it.  us for 7919 ragged tokens x 4096 channels of 16
// states, bf16, forward: 770 with a wave's channels to itself, 243 with the
// states in quarters, 147 with the outer products on the matrix cores and now.
#pragma once

#include <float.h>

#include "seed_channels.h"

namespace seed {
namespace channels {

constexpr int kWaves = 4;       // of a workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 8;        // tokens that go through LDS together
constexpr int kOwn = kTile / kWaves;   // of them prepared by one wave
// log2 of the tokens of a segment of the backward pass: 4 x 2048 tokens x 4096,
// bf16, 640 us then (64 tokens 661, 256 tokens 797), now 636; 3001 x 2050, fp32,
// 115 then (120, 204), now 110.
constexpr int kBackShift = 7;
constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147181f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|), and its slope,
// 1 / (1 + exp(-v)).  log(1 + e) = 2 atanh(e / (2 + e)): with s = e / (2 + e)
// at most 1/3, atanh(s) / s is a polynomial in s^2, here of degree 4 (fitted
// on Chebyshev points; 4e-9 of the value), so that small values keep their
// relative accuracy.
__device__ __forceinline__ float softplus_of(float v, float& e) {
  // (the constant in two parts: the first alone is 1.3e-8 short in every step)
  e = exp2_fast(-fmaf(fabsf(v), kLog2e, fabsf(v) * kLog2eRest));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
  float p = 0.14087337f;
  p = p * q + 0.139807165f;
  p = p * q + 0.20012425f;
  p = p * q + 0.333331585f;
  p = p * q + 1.f;
  return fmaxf(v, 0.f) + 2.f * s * p;
}
__device__ __forceinline__ float softplus_slope(float v, float e) {
  const float r = __builtin_amdgcn_rcpf(1.f + e);
  return v < 0.f ? e * r : r;
}
__device__ __forceinline__ float step_of(float v, bool softplus) {
  float e;
  return softplus ? softplus_of(v, e) : v;
}

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

// Nothing is moved over this point: what a token needs, in registers or on its
// way, does not pile up with the other tokens'.
__device__ __forceinline__ void next_token() { __builtin_amdgcn_sched_barrier(0); }
// ... and what these have come to is worked out here, not where it is used.
template <int Q>
__device__ __forceinline__ void settle(float (&x)[Q]) {
#pragma unroll
  for (int i = 0; i < Q; ++i) asm volatile("" : "+v"(x[i]));
}

// exp(delta A) = 2^(delta log2 e A): the steps are scaled, each with a rounding
// of its own, and not the rates, whose rounding would be the same in every
// factor of a product of decays.  The constant's own, 1.3e-8 of every exponent,
// is: of a product of decays it takes 1.3e-8 of its logarithm, a fifth of a
// rounding's half step.
__device__ __forceinline__ float in_powers_of_two(float delta) { return delta * kLog2e; }
// A rate of -infinity as the lowest number: a step above 2^-120 leaves nothing
// of a state then, as it would with -infinity, but a step of zero (a tile's
// tokens behind the sequence's end) leaves it as it is, where 0 (-infinity) is
// NaN.  One instruction, which keeps a NaN (a comparison and a choice cost the
// gradients two spilled registers, 627 us for 4 x 2048 x 4096 in place of 624).
__device__ __forceinline__ float rate_of(float A) { return __builtin_elementwise_maximum(A, -FLT_MAX); }
// A wave's rates as they lie in memory, and what they are taken as: the latter
// once the first tile's loads are sent, since it waits (16384 x 2048 in segments
// 259 us at the rates' load, 255 so).
template <int Q>
__device__ __forceinline__ void load_rates(const SelectArgs& a, const Mine& m, float (&A)[Q]) {
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int n = m.wave * Q + i;
    A[i] = n < a.d_state ? a.A[(size_t)m.c * a.d_state + n] : 0.f;
  }
}
template <int Q>
__device__ __forceinline__ void take_rates(float (&A)[Q]) {
  settle(A);
#pragma unroll
  for (int i = 0; i < Q; ++i) A[i] = rate_of(A[i]);
}

// 2^e h + x.  Where a state grows, e > 127, 2^e overflows before what it makes
// of a small h does, and is NaN with the zeros that h has before the first
// input: in two factors then, with h between them.  (2^254 h is infinite for
// every normal h, and so is 2^e h for e above.)
__device__ __forceinline__ float grown(float e, float h, float x) {
  const bool up = e > 127.f;
  return fmaf(exp2_fast(!up ? e : e < 254.f ? e - 127.f : 127.f), up ? 0x1p127f * h : h, x);
}
// Whether states can grow: a step that went through softplus is positive.
__device__ __forceinline__ bool may_grow(const SelectArgs& a, float A) { return !a.softplus || A > 0.f; }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= FLT_MAX; }

// The call's arguments, read again from where the launch put them: pointers and
// strides of a dozen arrays, each used once a tile, would take the scalar
// registers that the rows of B and C need.
typedef const __attribute__((address_space(4))) SelectArgs* ArgsAgain;
__device__ __forceinline__ ArgsAgain args_again() {
  auto p = (ArgsAgain)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// The rows of B and C: [token][group][wave][B of its Q states, C].
// C of the tokens of a tile for a wave's states, by scalar loads.  Tokens behind
// the last one of the sequence or segment take its row (their steps are zero,
// but a row of another sequence may hold an infinity).
typedef const __attribute__((address_space(4))) float* ScalarRow;
template <int Q>
struct ReadOuts {
  uintptr_t base;
  uint32_t step;
  int last;      // counted from the tile's first token
  __device__ __forceinline__ ReadOuts(const Mine& m, int t, int t1) : last(t1 - 1 - t) {
    const ArgsAgain a = args_again();
    base = (uintptr_t)(a->ws + a->at.rows) + (((size_t)t * a->groups + m.group) * 4 + m.wave) * (8 * Q) + 4 * Q;
    step = (uint32_t)a->groups * (32 * Q);
  }
  __device__ __forceinline__ ScalarRow operator[](int j) const {
    return (ScalarRow)(base + (uint32_t)(j < last ? j : last) * step);
  }
};

// The tile's rows in LDS: Q / 4 values a thread (Q = 2: one of every second).
template <int Q>
struct RowTile {
  static constexpr int kFloats = kTile * 8 * Q;
  float v[Q >= 4 ? Q / 4 : 1];
  __device__ __forceinline__ void load(int group, int t, int t1) {
    const ArgsAgain a = args_again();
    const float* rows = reinterpret_cast<const float*>(a->ws + a->at.rows);
#pragma unroll
    for (int q = 0; q < (kFloats + kThreads - 1) / kThreads; ++q) {
      const int at = (q * kThreads + (int)threadIdx.x) % kFloats, j = at / (8 * Q), in = at % (8 * Q);
      const size_t row = t + j < t1 ? t + j : t1 - 1;
      v[q] = rows[(row * a->groups + group) * (8 * Q) + in];
    }
  }
  __device__ __forceinline__ void store(float* lds) const {
#pragma unroll
    for (int q = 0; q < (kFloats + kThreads - 1) / kThreads; ++q)
      lds[(q * kThreads + (int)threadIdx.x) % kFloats] = v[q];
  }
};
// B (WHAT 0) or C (1) of token j for a wave's states, the same in every lane.
template <int Q, int WHAT>
__device__ __forceinline__ void row_values(const float* lds, const Mine& m, int j, float (&v)[Q]) {
  const float* p = lds + (j * kWaves + m.wave) * (2 * Q) + WHAT * Q;
  if constexpr (Q == 2) {
    load_vec<2>(p, v);
  } else {
#pragma unroll
    for (int q = 0; q < Q / 4; ++q) {
      const float4 x = reinterpret_cast<const float4*>(p)[q];
      v[4 * q] = x.x; v[4 * q + 1] = x.y; v[4 * q + 2] = x.z; v[4 * q + 3] = x.w;
    }
  }
}
// The same for outer products: a lane has those of state l % 4 of every four
// (Q = 2: all, for multiply-adds).
template <int Q, int WHAT>
struct Outer {
  float v[Q >= 4 ? Q / 4 : Q];
  __device__ __forceinline__ void load(const float* lds, const Mine& m, int j) {
    if constexpr (Q >= 4) {
      const float* p = lds + (j * kWaves + m.wave) * (2 * Q) + WHAT * Q + (__lane_id() & 3);
#pragma unroll
      for (int q = 0; q < Q / 4; ++q) v[q] = p[4 * q];
    } else {
      row_values<Q, WHAT>(lds, m, j, v);
    }
  }
};
// s + row x of a token: four states an instruction.
template <int Q, int WHAT>
__device__ __forceinline__ void add_outer(float (&s)[Q], const Outer<Q, WHAT>& o, float x) {
  if constexpr (Q >= 4) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int q = 0; q < Q / 4; ++q) {
      f32x4 acc = {s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]};
      acc = __builtin_amdgcn_mfma_f32_4x4x1f32(o.v[q], x, acc, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[4 * q + i] = acc[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < Q; ++i) s[i] += x * o.v[i];
  }
}
// A lane's value in row t of an array over tokens: the row's address is
// scalar, `at` the lane's bytes into it (channels are at most 2^20).
template <typename T>
__device__ __forceinline__ const T* in_row(const void* p, long long stride, int t, uint32_t at) {
  return reinterpret_cast<const T*>(static_cast<const char*>(p) + (long long)t * stride * (long long)sizeof(T) + at);
}
template <typename T>
__device__ __forceinline__ T* in_row(void* p, long long stride, int t, uint32_t at) {
  return reinterpret_cast<T*>(static_cast<char*>(p) + (long long)t * stride * (long long)sizeof(T) + at);
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
