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

// 16 columns of a bf16 array as raw accumulator tiles, rows from n on 0.
struct RawTiles {
  uint16_t x[4][4];
};
// p: the same address in every lane; `lane`: the lane's offset, 4 g rows and
// its column.
__device__ __forceinline__ RawTiles load_raw(const bf16_t* p, size_t ld, uint32_t lane, int n) {
  RawTiles v;
  if (n >= kC) {   // a whole chunk: no row to test
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bf16_t* row = p + (size_t)(16 * m + r) * ld;
        v.x[m][r] = row[lane];
      }
    return v;
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * m + 4 * (lane_id() >> 4) + r;
      const bf16_t* row = p + (size_t)(16 * m + r) * ld;
      v.x[m][r] = t < n ? row[lane] : 0;
    }
  return v;
}
__device__ __forceinline__ f32x4 tile_of(const RawTiles& v, int m) {
  f32x4 x;
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = bf16_bits_to_f32(v.x[m][r]);
  return x;
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

// Where a workgroup's columns are: grid n_seq * heads * (d_v / (16 NW)).
template <int NW>
struct Place {
  int seq, head, hk, col;
  __device__ __forceinline__ explicit Place(const ScanArgs& a) {
    const int blocks = a.d_v / (16 * NW);
    const int sh = blockIdx.x / blocks;
    seq = sh / a.heads;
    head = sh % a.heads;
    hk = head / (a.heads / a.key_heads);
    col = (blockIdx.x % blocks) * 16 * NW + (threadIdx.x >> 6) * 16 + (lane_id() & 15);
  }
};

}  // namespace scan
}  // namespace seed
