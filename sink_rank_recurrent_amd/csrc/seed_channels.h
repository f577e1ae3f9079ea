// Device helpers of the operators on channels: rows of fp32 and bf16 values,
// activations, and which tokens a piece of work covers.
#pragma once

#include "seed_channels_launch.h"
#include "seed_device.h"

namespace seed {
namespace channels {

// 1 / (1 + 2^(-x log2 e)) by the hardware's exponential and reciprocal (one
// ulp each; of the exponential the argument's rounding is at most |x| 2^-24, and
// the constant's, 1.3e-8 of itself, |x| 1.3e-8).
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// VW (1, 4 or 8) neighbouring values as they lie in memory, and as floats.
template <int VW, typename T>
struct Packed;
template <>
struct Packed<1, float> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void floats(float (&x)[1]) const { x[0] = v; }
  __device__ __forceinline__ void zero() { v = 0.f; }
  __device__ __forceinline__ void from(const float (&x)[1]) { v = x[0]; }
  __device__ __forceinline__ void store(float* p) const { *p = v; }
};
template <>
struct Packed<1, bf16_t> {
  bf16_t v;
  __device__ __forceinline__ void load(const bf16_t* p) { v = *p; }
  __device__ __forceinline__ void floats(float (&x)[1]) const { x[0] = bf16_bits_to_f32(v); }
  __device__ __forceinline__ void zero() { v = 0; }
  __device__ __forceinline__ void from(const float (&x)[1]) { v = (bf16_t)round_pair(x[0], 0.f); }
  __device__ __forceinline__ void store(bf16_t* p) const { *p = v; }
};
template <>
struct Packed<8, bf16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(u[j] << 16);
      x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void from(const float (&x)[8]) {
    v = make_uint4(round_pair(x[0], x[1]), round_pair(x[2], x[3]), round_pair(x[4], x[5]),
                   round_pair(x[6], x[7]));
  }
  __device__ __forceinline__ void store(bf16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
};
template <>
struct Packed<4, bf16_t> {
  uint2 v;
  __device__ __forceinline__ void load(const bf16_t* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void floats(float (&x)[4]) const {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  __device__ __forceinline__ void zero() { v = make_uint2(0, 0); }
  __device__ __forceinline__ void from(const float (&x)[4]) {
    v = make_uint2(round_pair(x[0], x[1]), round_pair(x[2], x[3]));
  }
  __device__ __forceinline__ void store(bf16_t* p) const { *reinterpret_cast<uint2*>(p) = v; }
};
// (float32: four values, 16 bytes)
template <>
struct Packed<4, float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void floats(float (&x)[4]) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void from(const float (&x)[4]) { v = make_float4(x[0], x[1], x[2], x[3]); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
};

// Tokens of a batch's sequences in runs of 2^shift: run c of sequence s has
// the number (first token of s >> shift) + s + c.  That needs no table and no
// synchronisation with the host, and gives every sequence at least one run,
// empty ones too; of a sequence's numbers the last may have no tokens.
struct Batch {
  const int* cu;
  int n_seq, tokens, len, shift;   // len: the equal lengths where cu is NULL
};
__host__ __device__ __forceinline__ Batch batch_of(const int* cu, int n_seq, int tokens, int shift) {
  return {cu, n_seq, tokens, cu ? 0 : tokens / n_seq, shift};
}
__device__ __forceinline__ int first_token(const Batch& b, int s) {
  const int at = b.cu ? b.cu[s] : s * b.len;
  return at < 0 ? 0 : at > b.tokens ? b.tokens : at;
}
__device__ __forceinline__ int first_run(const Batch& b, int s) { return (first_token(b, s) >> b.shift) + s; }

// The last sequence whose first run is `run` or before, by the whole wave (all
// 64 lanes, the same run).  64 sequences are looked at in one step.
__device__ __forceinline__ int sequence_of(const Batch& b, int run) {
  int base = 0, count = b.n_seq;
  while (count > 1) {
    const int step = (count + 63) >> 6, at = (int)__lane_id() * step;
    const bool there = at < count && first_run(b, base + at) <= run;
    const int last = __popcll(__ballot(there)) - 1, from = last > 0 ? last * step : 0;
    base += from;
    count = count - from < step ? count - from : step;
  }
  return __builtin_amdgcn_readfirstlane(base);
}

struct Run {
  int seq;
  int lo, hi;      // the sequence's tokens
  int t0, t1;      // the run's, t0 >= t1: none
  bool first;      // the sequence's first run
};
__device__ __forceinline__ Run run_of(const Batch& b, int seq, int run) {
  Run r;
  r.seq = seq;
  r.lo = first_token(b, seq);
  const int end = b.cu ? first_token(b, seq + 1) : r.lo + b.len;
  r.hi = end < r.lo ? r.lo : end;
  const long long c = (long long)run - ((r.lo >> b.shift) + seq);
  r.first = c == 0;
  const long long t0 = r.lo + (c < 0 ? r.hi : c << b.shift);   // no run of this sequence: no tokens
  r.t0 = t0 < r.hi ? (int)t0 : r.hi;
  r.t1 = r.hi - r.t0 > (1 << b.shift) ? r.t0 + (1 << b.shift) : r.hi;
  return r;
}

}  // namespace channels
}  // namespace seed
