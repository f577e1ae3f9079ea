// The gated linear recurrence over sequences, a chunk of 64 tokens at a time:
// device helpers and the arguments its kernels share.
//
// For one sequence and head, with S the state before the chunk, P_t the
// decay from the chunk's start through token t, F_t the decay after t to the
// chunk's end and G_ts the decay after s through t (products of the gates, so
// gates of 0 are exact; per key channel G_ts = P_t / P_s where that is safe):
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
// operand is the sum of three bf16 terms, each rounding what the ones before
// leave (2^-27 of it at last); the products whose weight is 2^-27 or less are
// left out, so a product of two fp32 operands takes six MFMAs, one with a bf16
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
constexpr int kRow = kC + 4;      // fp32 LDS rows of 64: 16-byte vectors, off the banks' stride
constexpr float kSafe = 0x1p-60f;  // the least decay (and 1 / the largest) of a chunk that is divided by
constexpr int kTriFrags = 6;      // fragments of a 64 x 64 triangle

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// One operand fragment in N bf16 terms, largest first.
template <int N>
struct Frag {
  u32x4 t[N];
};

// Two floats rounded to nearest bf16, in one word.
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// x as N bf16 terms, each what the ones before leave, rounded to nearest:
// N terms leave at most 2^-9N of x (nothing of a bf16 value).
template <int N>
__device__ __forceinline__ Frag<N> split(const float (&x)[8]) {
  Frag<N> f;
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t p = round_pair(r[2 * j], r[2 * j + 1]);
      f.t[n][j] = p;
      if (n + 1 < N) {
        r[2 * j] -= __uint_as_float(p << 16);
        r[2 * j + 1] -= __uint_as_float(p & 0xffff0000u);
      }
    }
  }
  return f;
}

// c += a b over the products of terms i, j with i + j < 3 (the smallest
// first).
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& c, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
  for (int o = 2; o >= 0; --o) {
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

__device__ __forceinline__ void store_scalar(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_scalar(bf16_t* p, float x) {
  *p = (bf16_t)round_pair(x, 0.f);
}

// Index of the fragment (row tile mt, contracted block ks) of a lower
// (upper) triangle of 64 x 64, -1 where the block is zero.
__host__ __device__ constexpr int lower_frag(int mt, int ks) {
  return mt < 2 ? (ks == 0 ? mt : -1) : 2 + 2 * (mt - 2) + ks;
}
__host__ __device__ constexpr int upper_frag(int mt, int ks) {
  return mt < 2 ? 2 * mt + ks : (ks == 1 ? 2 + mt : -1);
}

// A packed fragment of three terms, [frag][term][lane][8].
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

// The sequence of a slot, slots of `unit` tokens (start / unit + s the first
// of sequence s): the last whose first slot is not behind it; a wave tries 64
// at a time.
struct Found {
  int seq;
  Range rg;
};
__device__ __forceinline__ Found sequence_of_slot(const ScanArgs& a, int slot, int unit) {
  const int lane = threadIdx.x & 63;
  int lo = 0, span = a.n_seq;
  Range r;
  for (;;) {
    const int step = (span + 63) >> 6;
    const int i = min(lo + lane * step, a.n_seq - 1);
    r = sequence(a, i);
    const bool at = lane * step < span && r.start / unit + i <= slot;
    const int last = 63 - __builtin_clzll(__ballot(at) | 1);
    lo += last * step;
    if (step == 1) {
      return {__builtin_amdgcn_readfirstlane(lo),
              {__builtin_amdgcn_readlane(r.start, last), __builtin_amdgcn_readlane(r.len, last)}};
    }
    span = min(step, span - last * step);
  }
}

// The head of number x of a token's: heads in turn over the key heads, so that
// (with workgroups dealt to 8 XCDs in turn) heads that share keys share an
// L2.  Kernels count heads fastest: workgroups that run together then read
// whole rows (one head at a time, preparation of 64 x 512 tokens x 16 heads
// took 8 % longer, the KDA gradients 22 %).
__device__ __forceinline__ int head_of(const ScanArgs& a, int x) {
  return x % a.key_heads * (a.heads / a.key_heads) + x / a.key_heads;
}

// The chunk of a slot: sequence and first token, n tokens (0: none).
struct Chunk {
  int seq, tok, n, index;
};
__device__ __forceinline__ Chunk chunk_of_slot(const ScanArgs& a, int slot) {
  const Found found = sequence_of_slot(a, slot, kC);
  const int lo = found.seq;
  const Range r = found.rg;
  const int c = slot - slot_base(r, lo);
  if (c < 0 || c * kC >= r.len) return {lo, 0, 0, 0};
  const int left = r.len - c * kC;
  return {lo, r.start + c * kC, left < kC ? left : kC, c};
}

// ---------------------------------------------------------------------------
// A 64 x DK operand in LDS: one bf16 plane per term, rows of DK / 8 pieces of
// 16 bytes.  Piece c of row t lies at c ^ swizzle(t): the 16 rows a fragment
// reads at one c then cover all 64 banks.
template <int DK>
__device__ __forceinline__ int swizzle(int t) {
  return DK == 128 ? t & 15 : (t >> 1) & 7;
}
template <int DK>
__device__ __forceinline__ int piece_at(int t, int c) {   // in bytes
  return t * (DK * 2) + ((c ^ swizzle<DK>(t)) << 4);
}
template <int DK>
constexpr int kPlane = kC * DK * 2;   // bytes

// The channel of row 4 g + r of state tile m.  Tiles 2 ks and 2 ks + 1 hold
// channels 32 ks + 8 g + 0..7 in a lane, so that the state's fragments
// contract over 16-byte pieces of K's rows.
__device__ __forceinline__ int state_row(int m) {
  return 32 * (m >> 1) + 8 * (lane_id() >> 4) + 4 * (m & 1);
}

// Rows 16 mt .. + 15 as a fragment, contracted over channels 32 ks .. + 31.
template <int DK, int N>
__device__ __forceinline__ Frag<N> lds_rows(const char* planes, int mt, int ks) {
  const int l = lane_id(), at = piece_at<DK>(16 * mt + (l & 15), 4 * ks + (l >> 4));
  Frag<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.t[n] = *reinterpret_cast<const u32x4*>(planes + n * kPlane<DK> + at);
  return f;
}

// The transpose: state tile m's channels as rows, contracted over tokens
// 32 ks .. + 31 in accumulator order, by transposing LDS reads (a block of
// 16 lanes reads 4 rows of 16 values, lane i gets the 4 of column i).
template <int DK, int N>
__device__ __forceinline__ Frag<N> lds_cols(const char* planes, int m, int ks) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const int l = lane_id(), i = l & 15, g = l >> 4;
  Frag<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = 32 * ks + 16 * h + 4 * g + (i >> 2);
      const char* at = planes + n * kPlane<DK> + piece_at<DK>(t, 4 * (m >> 1) + (i & 3)) + 8 * (m & 1);
      const u32x2 x = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                     (__attribute__((address_space(3))) bf16x4*)(at)));
      f.t[n][2 * h] = x[0];
      f.t[n][2 * h + 1] = x[1];
    }
  return f;
}

// The transpose with the channels 16 m .. + 15 in their own order.
template <int DK, int N>
__device__ __forceinline__ Frag<N> lds_channels(const char* planes, int m, int ks) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const int l = lane_id(), i = l & 15, g = l >> 4;
  Frag<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = 32 * ks + 16 * h + 4 * g + (i >> 2);
      const char* at = planes + n * kPlane<DK> + piece_at<DK>(t, 2 * m + ((i & 3) >> 1)) + 8 * (i & 1);
      const u32x2 x = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                     (__attribute__((address_space(3))) bf16x4*)(at)));
      f.t[n][2 * h] = x[0];
      f.t[n][2 * h + 1] = x[1];
    }
  return f;
}

// One fragment of a pack in LDS ([frag][term][lane][8]).
template <int N>
__device__ __forceinline__ Frag<N> lds_pack(const char* pack, int frag) {
  Frag<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n)
    f.t[n] = *reinterpret_cast<const u32x4*>(pack + (frag * N + n) * (kFrag * 2) + lane_id() * 16);
  return f;
}

// Global memory to LDS without registers: 16 bytes a lane from `from` (the
// same in every lane) + `off`, to 64 consecutive places from LDS offset `to`
// (the same in every lane).  Written as asm because the compiler would make
// every later LDS read wait for it, another buffer's too; the caller waits
// (async_wait, then a barrier).  M0 holds the LDS side and is put back for the
// compiler.  The compiler fills no wait states inside asm: the two moves and
// s_nop 2 are the five that a memory instruction needs behind a vector
// instruction that wrote its scalar base (the readfirstlanes above), and the
// one behind the write of M0.
__device__ __forceinline__ void async_copy(const void* from, uint32_t off, uint32_t to) {
  uint32_t kept;
  const uint64_t p = reinterpret_cast<uint64_t>(from);
  const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(p >> 32)) << 32 |
                        (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)p);
  to = __builtin_amdgcn_readfirstlane(to);
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 2\n\t"
               "global_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
               : "=&s"(kept) : "v"(off), "s"(base), "s"(to) : "memory");
}
__device__ __forceinline__ void async_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_offset(const char* p) {
  return __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p);
}
// The wave's number in its workgroup, as a scalar.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// A chunk's rows of bf16 arrays [tokens][heads][DK] (K, and Q if it has a
// place) into planes, W waves together; rows from n on repeat row n - 1.
// ld: elements from row to row.
template <int DK, int W>
__device__ __forceinline__ void async_rows(const bf16_t* K, const bf16_t* Q, uint32_t ld, int n,
                                           uint32_t k_to, uint32_t q_to, bool has_q, int wave) {
  constexpr int PR = DK / 8, PER = 64 / PR;   // pieces a row, rows a step
#pragma unroll
  for (int j = 0; j < kC / PER / W; ++j) {
    const int i = wave + j * W, t = i * PER + lane_id() / PR;
    const int c = (lane_id() % PR) ^ swizzle<DK>(t);
    const uint32_t off = (uint32_t)min(t, n - 1) * (2 * ld) + 16 * c;
    async_copy(K, off, k_to + i * 1024);
    if (has_q) async_copy(Q, off, q_to + i * 1024);
  }
}

// A pack's fragments.
template <int W>
__device__ __forceinline__ void async_pack(const uint16_t* pack, uint32_t to, int wave) {
#pragma unroll
  for (int j = 0; j < (kTriFrags * 3 + W - 1) / W; ++j) {
    const int i = wave + j * W;
    if (i < kTriFrags * 3) async_copy(pack + i * kFrag, lane_id() * 16, to + i * 1024);
  }
}

// Eight channels from col0 + 8 g of a row.
template <typename T>
__device__ __forceinline__ void load_piece(const T* __restrict__ row, int col0, bool live,
                                           float (&x)[8]) {
  const int g = lane_id() >> 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = 0.f;
  if constexpr (sizeof(T) == 2) {
    if (live) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(row + col0 + 8 * g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(v[j] << 16);
        x[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
      }
    }
  } else if (live) {
    float a[4], b[4];
    load_vec<4>(row + col0 + 8 * g, a);
    load_vec<4>(row + col0 + 8 * g + 4, b);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = a[r];
      x[4 + r] = b[r];
    }
  }
}

// Decay factors of a chunk for scalar gates, for pairs in different blocks
// of 16: G_ts = pre[t] mid[block t][block s] suf[s], pre from t's block's
// start through t, suf behind s to its block's end; within a block, G_ts is
// multiplied up (inside).
struct __attribute__((aligned(16))) Decay {
  float gate[kC + 4], pre[kC], suf[kC], mid[16];   // gate: read 3 past a block
};
// The decay behind s through t of one block, and (rows: along t, else along
// s) of the three tokens that follow it in a lane.
template <bool ROWS>
__device__ __forceinline__ f32x4 inside(const float* gate, int t, int s) {
  const float* g = gate + (t & ~15);
  t &= 15;
  s &= 15;
  const int last = ROWS ? s : s + 3;   // the pair with the shortest stretch
  float x = 1.f;
#pragma unroll
  for (int o = 1; o < 16; ++o) {
    const float y = g[o];
    x *= o > last && o <= t ? y : 1.f;
  }
  f32x4 out;
  if (ROWS) {
    out[0] = x;
#pragma unroll
    for (int r = 1; r < 4; ++r) {
      const float y = g[t + r];
      out[r] = out[r - 1] * (t + r > s ? y : 1.f);
    }
  } else {
    out[3] = x;
#pragma unroll
    for (int r = 2; r >= 0; --r) {
      const float y = g[s + r + 1];
      out[r] = out[r + 1] * (s + r < t ? y : 1.f);
    }
  }
  return out;
}
// One wave; lane l holds gate l.  P and F of token l come back.
__device__ __forceinline__ void decays(Decay& d, float gate, float& P, float& F) {
  const int l = lane_id(), l16 = l & 15;
  float p = gate, s = gate;
#pragma unroll
  for (int o = 1; o < 16; o *= 2) {
    const float x = __shfl_up(p, o), y = __shfl_down(s, o);
    p *= l16 >= o ? x : 1.f;
    s *= l16 + o < 16 ? y : 1.f;
  }
  const float next = __shfl_down(s, 1);
  s = l16 == 15 ? 1.f : next;   // behind l only
  const float t0 = __shfl(p, 15), t1 = __shfl(p, 31), t2 = __shfl(p, 47), t3 = __shfl(p, 63);
  d.gate[l] = gate;
  d.pre[l] = p;
  d.suf[l] = s;
  if (l < 16) {
    const int a = l >> 2, b = l & 3;   // blocks between b and a
    d.mid[l] = (b < 1 && a > 1 ? t1 : 1.f) * (b < 2 && a > 2 ? t2 : 1.f);
  }
  const int blk = l >> 4;
  P = p * (blk > 0 ? t0 : 1.f) * (blk > 1 ? t1 : 1.f) * (blk > 2 ? t2 : 1.f);
  F = s * (blk < 1 ? t1 : 1.f) * (blk < 2 ? t2 : 1.f) * (blk < 3 ? t3 : 1.f);
}

// c[m] += a[m] b for MT row tiles, the tiles in turn so that consecutive
// MFMAs do not wait for each other.
template <int MT, int NA, int NB>
__device__ __forceinline__ void mma_tiles(f32x4 (&c)[MT], const Frag<NA> (&a)[MT],
                                          const Frag<NB>& b) {
#pragma unroll
  for (int o = 2; o >= 0; --o) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = o - i;
      if (j < 0 || j >= NB) continue;
#pragma unroll
      for (int m = 0; m < MT; ++m)
        c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[m].t[i]),
                                                       __builtin_bit_cast(bf16x8, b.t[j]), c[m], 0, 0, 0);
    }
  }
}

}  // namespace scan
}  // namespace seed
