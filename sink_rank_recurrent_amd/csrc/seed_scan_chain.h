// What the kernels that go from chunk to chunk share: a wave's 16 columns of
// the state and of the chunk's rows, as accumulator tiles.
#pragma once

#include "seed_scan.h"

namespace seed {
namespace scan {

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

template <int N>
__device__ __forceinline__ Frag<N> split_tiles(const f32x4& a, const f32x4& b) {
  float x[8];
  tiles_to_floats(a, b, x);
  return split<N>(x);
}

// Rows 16 m + 4 g + r of a 64-vector in LDS.
__device__ __forceinline__ f32x4 lds_vec(const char* vec, int m) {
  return *reinterpret_cast<const f32x4*>(vec + 64 * m + 16 * (lane_id() >> 4));
}

// A wave's 64 rows x 16 columns of an array, in LDS of its own (bf16: 2 KB,
// rows of 32 bytes; float32: 4 KB).  Loads repeat row n - 1 from row n on, and
// first wait for the wave's reads of what they replace.
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
template <typename T>
constexpr int kOwn = kC * 16 * (int)sizeof(T);
__device__ __forceinline__ void wave_load(const float* p, uint32_t ld, int n, uint32_t to) {
  lds_done();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 16 * i + (lane_id() >> 2);
    async_copy(p, (uint32_t)min(t, n - 1) * (4 * ld) + 16 * (lane_id() & 3), to + 1024 * i);
  }
}
__device__ __forceinline__ void wave_load(const bf16_t* p, uint32_t ld, int n, uint32_t to) {
  lds_done();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 32 * i + (lane_id() >> 1);
    async_copy(p, (uint32_t)min(t, n - 1) * (2 * ld) + 16 * (lane_id() & 1), to + 1024 * i);
  }
}
template <typename T>
__device__ __forceinline__ f32x4 wave_tile(const char* from, int m);
template <>
__device__ __forceinline__ f32x4 wave_tile<float>(const char* from, int m) {
  const float* at = reinterpret_cast<const float*>(from) + (16 * m + 4 * (lane_id() >> 4)) * 16 + (lane_id() & 15);
  return f32x4{at[0], at[16], at[32], at[48]};
}
// As accumulator tiles, by transposing reads.
template <>
__device__ __forceinline__ f32x4 wave_tile<bf16_t>(const char* from, int m) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const int l = lane_id(), i = l & 15, g = l >> 4;
  const char* at = from + (16 * m + 4 * g + (i >> 2)) * 32 + 8 * (i & 3);
  const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                                                (__attribute__((address_space(3))) bf16x4*)(at)));
  return f32x4{__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u),
               __uint_as_float(x[1] << 16), __uint_as_float(x[1] & 0xffff0000u)};
}
// Accumulator tiles out through the same place: rows of 16 bytes a lane.
__device__ __forceinline__ void wave_store(bf16_t* p, size_t ld, int n, const f32x4 (&x)[4], char* by) {
  const int l = lane_id();
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<bf16_t*>(by + (16 * m + 4 * (l >> 4) + r) * 32 + 2 * (l & 15)) =
          (bf16_t)round_pair(x[m][r], 0.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 32 * i + (l >> 1);
    const u32x4 v = *reinterpret_cast<const u32x4*>(by + 1024 * i + 16 * l);
    if (t < n) *reinterpret_cast<u32x4*>(p + (size_t)t * ld + 8 * (l & 1)) = v;
  }
}
__device__ __forceinline__ void wave_store(float* p, size_t ld, int n, const f32x4 (&x)[4], char* by) {
  const int l = lane_id();
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      reinterpret_cast<float*>(by)[(16 * m + 4 * (l >> 4) + r) * 16 + (l & 15)] = x[m][r];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 16 * i + (l >> 2);
    const f32x4 v = *reinterpret_cast<const f32x4*>(by + 1024 * i + 16 * l);
    if (t < n) *reinterpret_cast<f32x4*>(p + (size_t)t * ld + 4 * (l & 3)) = v;
  }
}
template <typename T>
__device__ __forceinline__ void store_tiles(T* p, size_t ld, uint32_t lane, int n,
                                            const f32x4 (&x)[4]) {
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * m + 4 * (lane_id() >> 4) + r;
      T* row = p + (size_t)(16 * m + r) * ld;
      if (t < n) store_scalar(row + lane, x[m][r]);
    }
}
// The same for the fp32 arrays of the workspace (every row) and for states
// (rows in the order of state_row; `lane` 8 g rows and the column).
__device__ __forceinline__ void keep_tiles(float* p, int ld, uint32_t lane, const f32x4 (&x)[4]) {
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float* row = p + (16 * m + r) * ld;
      row[lane] = x[m][r];
    }
}
template <int IT>
__device__ __forceinline__ void keep_state(float* p, int ld, uint32_t lane, const f32x4 (&x)[IT]) {
#pragma unroll
  for (int m = 0; m < IT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float* row = p + (32 * (m >> 1) + 4 * (m & 1) + r) * ld;
      row[lane] = x[m][r];
    }
}
// A chunk's state in the workspace, in the order the waves hold it: 16
// columns, then their tiles, 1 KB each.
template <int IT>
__device__ __forceinline__ void keep_chunk_state(float* p, int col0, const f32x4 (&x)[IT]) {
#pragma unroll
  for (int m = 0; m < IT; ++m)
    *reinterpret_cast<f32x4*>(p + (col0 / 16 * IT + m) * 256 + lane_id() * 4) = x[m];
}
// Four channels of state_row(m) of lanes 16 g .., column j, of such a state.
template <int DK>
__device__ __forceinline__ int chunk_state_at(int m, int g, int j) {
  return ((j >> 4) * (DK / 16) + m) * 256 + (16 * g + (j & 15)) * 4;
}
template <int IT>
__device__ __forceinline__ void load_state(const float* p, int ld, uint32_t lane, f32x4 (&x)[IT]) {
#pragma unroll
  for (int m = 0; m < IT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float* row = p ? p + (32 * (m >> 1) + 4 * (m & 1) + r) * ld : nullptr;
      x[m][r] = p ? row[lane] : 0.f;
    }
}
// Rows from n on are no tokens: their results are dropped.
__device__ __forceinline__ void drop_rows(f32x4 (&x)[4], int n) {
  if (n < kC) {
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (16 * m + 4 * (lane_id() >> 4) + r >= n) x[m][r] = 0.f;
  }
}

// Eight values of an array as loaded.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + 4);
  }
  __device__ __forceinline__ void clear() { a = b = zero4(); }
  __device__ __forceinline__ void get(float (&x)[8]) const { tiles_to_floats(a, b, x); }
};
template <>
struct Piece<bf16_t> {
  u32x4 a;
  __device__ __forceinline__ void load(const bf16_t* p) { a = *reinterpret_cast<const u32x4*>(p); }
  __device__ __forceinline__ void clear() { a = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(a[j] << 16);
      x[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  }
};

// What a workgroup walks: 16 NW columns of a head's state (of `columns` in
// all) through chunks c0 .. c1 - 1 of a sequence: all of them, or a segment.
// A wave whose columns are d_v and more carries columns of the unit matrix
// instead of the state's, with V = 0.  c0 > c1: nothing.
template <int NW>
struct Walk {
  int seq, head, hk, col0, col, c0, c1, chunks, base;   // col0: the wave's first column
  size_t segment;                                       // (segment, head), for what is kept for it
  Range rg;
  // the sequence has several segments: all take their first states from the
  // workspace, since S may be S0 (dS0 may be dS), written by one workgroup
  // while another has yet to start
  bool split;
  __device__ __forceinline__ Walk(const ScanArgs& a, int columns) {
    const int blocks = columns / (16 * NW);
    const int sh = blockIdx.x / blocks;
    const int first = sh / a.heads;
    head = head_of(a, sh % a.heads);
    segment = (size_t)first * a.heads + head;
    if (a.at.seg) {
      const Found found = sequence_of_slot(a, first, kC * a.at.seg);
      seq = found.seq;
      rg = found.rg;
    } else {
      seq = first;
      rg = sequence(a, seq);
    }
    chunks = (rg.len + kC - 1) / kC;
    base = slot_base(rg, seq);
    c0 = 0;
    c1 = chunks;
    split = a.at.seg > 0 && chunks > a.at.seg;
    if (a.at.seg) {
      const int i = first - (rg.start / (kC * a.at.seg) + seq);
      c0 = i * a.at.seg;
      c1 = min(chunks, c0 + a.at.seg);
      if (i < 0 || (i > 0 && c0 >= chunks)) c0 = c1 + 1;
    }
    hk = head / (a.heads / a.key_heads);
    col0 = (blockIdx.x % blocks) * 16 * NW + wave_id() * 16;
    col = col0 + (lane_id() & 15);
  }
};
inline size_t walk_grid(const ScanArgs& a, int columns, int waves) {
  return (size_t)(a.at.seg ? a.at.segs : a.n_seq) * a.heads * (columns / (16 * waves));
}

// A kept state in the waves' order, back into them.
template <int IT>
__device__ __forceinline__ void load_chunk_state(const float* p, int col0, f32x4 (&x)[IT]) {
#pragma unroll
  for (int m = 0; m < IT; ++m)
    x[m] = *reinterpret_cast<const f32x4*>(p + (col0 / 16 * IT + m) * 256 + lane_id() * 4);
}
// Columns of the unit matrix.
template <int IT>
__device__ __forceinline__ void unit_state(int col, f32x4 (&x)[IT]) {
#pragma unroll
  for (int m = 0; m < IT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) x[m][r] = state_row(m) + r == col ? 1.f : 0.f;
}

enum WalkMode { kRead = 0, kSave = 1, kCarry = 2 };

// Waves of a workgroup: all of a head's columns, or half of 128 where whole
// heads would leave some of the 256 CUs idle (64 x 32 chunks of 128 x 128 GDN
// heads: backward 207 us with four waves, 236 with eight, forward 126 and 154;
// forward of 1024 x 8 chunks: 391 us with four, 298 with eight).
inline int walk_waves(const ScanArgs& a) {
  const int all = a.d_v / 16;
  return all == 8 && (a.at.seg || (long long)a.n_seq * a.heads < 256) ? 4 : all;
}

}  // namespace scan
}  // namespace seed
