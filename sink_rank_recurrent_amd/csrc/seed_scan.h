// The gated linear recurrence over sequences, a chunk of 64 tokens at a time:
// device helpers and the arguments its kernels share.
//
// For one sequence and head, with S the state before the chunk, P_t the
// decay from the chunk's start through token t, F_t the decay after t to the
// chunk's end and G_ts the decay after s through t (products of the gates,
// never quotients, so gates of 0 are exact):
//   L_ts = G_ts k_t.k_s (s < t),  M_ts = G_ts q_t.k_s (s <= t)
//   R = V - P (K S),   E = R - N (beta R),  N = (I + L beta)^-1 L,
//   u = beta E  (Mamba-2: u = E = V),
//   O = P (Q S) + M u,   S' = P_end S + (F K)^T u
// and backwards, with H the gradient of S':
//   dU = M^T dO + F (K H),  Y = dU - N^T (beta dU),  dV = dR = beta Y,
//   dbeta = Y.E,  dS = P_end H + (P Q)^T dO - (P K)^T dR
//   dQ = P (dO S^T) + (dM G) K,          dM = dO u^T (s <= t)
//   dK = F (u H^T) - P (dR S^T) + (dL G) K + (dL G)^T K + (dM G)^T Q,
//                                        dL = -dR u^T (s < t).
//
// Arithmetic: v_mfma_f32_16x16x32_bf16 with fp32 accumulators.  An fp32
// operand is the exact sum of three bf16 terms (its 24 significant bits cut
// into three times 8); the products whose weight is 2^-24 or less are left
// out, so a product of two fp32 operands takes six MFMAs, one with a bf16
// input three.
#pragma once

#include "seed_device.h"
#include "seed_sequence_launch.h"

namespace seed {
namespace scan {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kC = kScanChunk;
constexpr int kFrag = 512;        // bf16 values of one 16 x 32 operand fragment
constexpr int kTriFrags = 6;      // fragments of a 64 x 64 triangle

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// One operand fragment in N bf16 terms, largest first.
template <int N>
struct Frag {
  u32x4 t[N];
};

__device__ __forceinline__ uint32_t pack_hi(float lo, float hi) {
  // the upper halves of two floats in one word
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

__device__ __forceinline__ float cut(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}

// x as N truncated bf16 terms: exact for N = 3 (and for bf16 values with
// N = 1); N = 2 leaves at most 2^-16 of x.
template <int N>
__device__ __forceinline__ Frag<N> split(const float (&x)[8]) {
  Frag<N> f;
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.t[n][j] = pack_hi(r[2 * j], r[2 * j + 1]);
    if (n + 1 < N) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] -= cut(r[j]);
    }
  }
  return f;
}

// c += a b over the products of terms i, j with i + j < ORDER (the smallest
// first).
template <int NA, int NB, int ORDER = 3>
__device__ __forceinline__ void mma(f32x4& c, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
  for (int o = ORDER - 1; o >= 0; --o) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = o - i;
      if (j >= 0 && j < NB)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.t[i]),
                                                    __builtin_bit_cast(bf16x8, b.t[j]), c, 0, 0, 0);
    }
  }
}

// Fragment order of the contracted index.  Lane l holds row (or column)
// l % 16 and, in slots j = 0..7, the indices 16 (j / 4) + 4 (l / 16) + j % 4
// of the fragment's 32: the order in which two 16 x 16 accumulator tiles
// hold their rows, so that a result feeds the next product as its right
// operand without leaving the registers.
__device__ __forceinline__ void tiles_to_floats(const f32x4& a, const f32x4& b, float (&x)[8]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    x[r] = a[r];
    x[4 + r] = b[r];
  }
}

// Rows of a row-major array (ld elements a row) as a fragment: row = the
// lane's, the contracted index along the row from `col0`.
template <typename T>
__device__ __forceinline__ void load_row8(const T* __restrict__ row, int col0, bool live,
                                          float (&x)[8]) {
  const int g = lane_id() >> 4;
  if (live) {
    float a[4], b[4];
    load_vec<4>(row + col0 + 4 * g, a);
    load_vec<4>(row + col0 + 16 + 4 * g, b);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = a[r];
      x[4 + r] = b[r];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.f;
  }
}

// A column of a row-major array as a fragment: the contracted index runs
// over rows row0 .. row0 + 31, of which `rows` are live.
template <typename T>
__device__ __forceinline__ void load_col8(const T* __restrict__ base, size_t ld, int row0,
                                          int rows, float (&x)[8]) {
  const int g = lane_id() >> 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int t = row0 + 16 * (j >> 2) + 4 * g + (j & 3);
    x[j] = t < rows ? load_scalar(base + (size_t)t * ld) : 0.f;
  }
}

__device__ __forceinline__ void store_scalar(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_scalar(bf16_t* p, float x) {
  *p = (bf16_t)round_nearest16<kStoreBF16>(x);
}

// Index of the fragment (row tile mt, contracted block ks) of a lower
// (upper) triangle of 64 x 64, -1 where the block is zero.
__host__ __device__ constexpr int lower_frag(int mt, int ks) {
  return mt < 2 ? (ks == 0 ? mt : -1) : 2 + 2 * (mt - 2) + ks;
}
__host__ __device__ constexpr int upper_frag(int mt, int ks) {
  return mt < 2 ? 2 * mt + ks : (ks == 1 ? 2 + mt : -1);
}

// A packed fragment of three terms: [frag][term][lane][8].
__device__ __forceinline__ Frag<3> load_pack(const uint16_t* __restrict__ pack, int frag) {
  Frag<3> f;
#pragma unroll
  for (int n = 0; n < 3; ++n)
    f.t[n] = *reinterpret_cast<const u32x4*>(pack + (size_t)(frag * 3 + n) * kFrag + lane_id() * 8);
  return f;
}
__device__ __forceinline__ void store_pack(uint16_t* __restrict__ pack, int frag,
                                           const Frag<3>& f) {
#pragma unroll
  for (int n = 0; n < 3; ++n)
    *reinterpret_cast<u32x4*>(pack + (size_t)(frag * 3 + n) * kFrag + lane_id() * 8) = f.t[n];
}

// Sequence s: its first token and length.  Offsets that do not rise, or
// leave 0 .. tokens, give wrong results but no access outside the arrays.
struct Range {
  int start, len;
};
__device__ __forceinline__ Range sequence(const ScanArgs& a, int s) {
  if (a.cu == nullptr) {
    const int len = a.tokens / a.n_seq;
    return {s * len, len};
  }
  int b = a.cu[s], e = a.cu[s + 1];
  b = b < 0 ? 0 : b > a.tokens ? a.tokens : b;
  e = e < b ? b : e > a.tokens ? a.tokens : e;
  return {b, e - b};
}

// Chunk c of sequence s has slot start / 64 + s + c of the workspace: rising
// in s, disjoint, and below tokens / 64 + n_seq, without a table.
__device__ __forceinline__ int slot_base(const Range& r, int s) { return r.start / kC + s; }

// The chunk of a slot: sequence and first token, n tokens (0: none).
struct Chunk {
  int seq, tok, n, index;
};
__device__ __forceinline__ Chunk chunk_of_slot(const ScanArgs& a, int slot) {
  int lo = 0, hi = a.n_seq - 1;   // the last sequence whose base is <= slot
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (slot_base(sequence(a, mid), mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const Range r = sequence(a, lo);
  const int c = slot - slot_base(r, lo);
  if (c < 0 || c * kC >= r.len) return {lo, 0, 0, 0};
  const int left = r.len - c * kC;
  return {lo, r.start + c * kC, left < kC ? left : kC, c};
}

}  // namespace scan
}  // namespace seed
