// The states at the starts of a sequence's segments, from what each segment
// makes of zero (N) and of the unit matrix (A): S' = A S + N, one after the
// other; backwards the gradients at their ends, H = A^T H' + G.  The waves
// own 16 columns as everywhere; A goes through LDS in three bf16 terms, the
// next one's values loaded meanwhile.  (Mamba-2: A is a factor.)  A chain of
// one 64 x 64 or 128 x 128 product a segment, bound by its latency: 16 heads x
// 16 segments of 64 x 64 take 37 us.
#include "seed_scan_chain.h"

namespace seed {
namespace scan {
namespace {

template <int DK>
constexpr int kCarryPlane = DK * DK * 2;   // bytes of one term of A

// Rows k, pieces of 8 channels.  Forward, channels are rows of the result and
// k is contracted; backward the other way round.
template <int DK>
__device__ __forceinline__ Frag<3> carry_rows(const char* planes, int m, int ks) {   // A
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const int l = lane_id(), i = l & 15, g = l >> 4;
  Frag<3> f;
#pragma unroll
  for (int n = 0; n < 3; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 32 * ks + 8 * g + 4 * h + (i >> 2);
      const char* at = planes + n * kCarryPlane<DK> + piece_at<DK>(k, 4 * (m >> 1) + (i & 3)) + 8 * (m & 1);
      const u32x2 x = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                     (__attribute__((address_space(3))) bf16x4*)(at)));
      f.t[n][2 * h] = x[0];
      f.t[n][2 * h + 1] = x[1];
    }
  return f;
}
template <int DK>
__device__ __forceinline__ Frag<3> carry_cols(const char* planes, int m, int ks) {   // A^T
  const int l = lane_id(), i = l & 15, g = l >> 4;
  const int k = 32 * (m >> 1) + 8 * (i >> 2) + 4 * (m & 1) + (i & 3);
  Frag<3> f;
#pragma unroll
  for (int n = 0; n < 3; ++n)
    f.t[n] = *reinterpret_cast<const u32x4*>(planes + n * kCarryPlane<DK> + piece_at<DK>(k, 4 * ks + g));
  return f;
}

// grid: n_seq * heads * (d_v / 64), four waves.
template <int DK, bool DELTA, bool BACK>
__global__ __launch_bounds__(256) void join_kernel(ScanArgs a) {
  constexpr int IT = DK / 16, SHARE = DELTA ? DK * DK / 8 / 256 : 1;   // pieces of A a thread
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int blocks = a.d_v / 64, sh = blockIdx.x / blocks, seq = sh / a.heads, head = sh % a.heads;
  const int col0 = (blockIdx.x % blocks) * 64 + wave_id() * 16, col = col0 + (lane_id() & 15);
  const Range rg = sequence(a, seq);
  const int chunks = (rg.len + kC - 1) / kC, seg = a.at.seg;
  const int segments = (chunks + seg - 1) / seg, base = rg.start / (kC * seg) + seq;
  if (segments < 2) return;
  const float* trans = reinterpret_cast<const float*>(a.ws + a.at.trans);
  const float* carry = reinterpret_cast<const float*>(a.ws + a.at.carry);
  float* start = reinterpret_cast<float*>(a.ws + a.at.start);
  const size_t size = (size_t)DK * a.d_v;
  auto unit = [&](int i) { return (size_t)(base + i) * a.heads + head; };

  // a thread's pieces of A: column k, channels 32 mp + 8 g .. + 7
  f32x4 lo[SHARE], hi[SHARE];
  auto fetch = [&](int i) {
#pragma unroll
    for (int j = 0; j < SHARE; ++j) {
      const int e = j * 256 + threadIdx.x, k = e / (DK / 8), c = e % (DK / 8);
      const float* p = trans + unit(i) * DK * DK;
      lo[j] = *reinterpret_cast<const f32x4*>(p + chunk_state_at<DK>(2 * (c >> 2), c & 3, k));
      hi[j] = *reinterpret_cast<const f32x4*>(p + chunk_state_at<DK>(2 * (c >> 2) + 1, c & 3, k));
    }
  };
  f32x4 S[IT];
  const size_t state = ((size_t)seq * a.heads + head) * size;
  const float* from = BACK ? a.dS : a.S0;
  load_state(from ? from + state : nullptr, a.d_v, 8 * (lane_id() >> 4) * a.d_v + col, S);
  const int first = BACK ? segments - 1 : 0;
  keep_chunk_state(start + unit(first) * size, col0, S);
  if (DELTA && !BACK) fetch(first);
  for (int n = 0; n + 1 < segments; ++n) {
    const int i = BACK ? segments - 1 - n : n;   // the segment passed through
    f32x4 x[IT];
    load_chunk_state(carry + unit(i) * size, col0, x);
    if (BACK && n == 0) {   // the last segment's carry already has dS
#pragma unroll
      for (int m = 0; m < IT; ++m) S[m] = x[m];
    } else if (DELTA) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < SHARE; ++j) {
        const int e = j * 256 + threadIdx.x, k = e / (DK / 8), c = e % (DK / 8);
        float y[8];
        tiles_to_floats(lo[j], hi[j], y);
        const Frag<3> f = split<3>(y);
#pragma unroll
        for (int t = 0; t < 3; ++t)
          *reinterpret_cast<u32x4*>(lds + t * kCarryPlane<DK> + piece_at<DK>(k, c)) = f.t[t];
      }
      __syncthreads();
    } else {
      const float f = trans[unit(i)];
#pragma unroll
      for (int m = 0; m < IT; ++m) S[m] = f * S[m] + x[m];
    }
    if (DELTA && n + 2 < segments) fetch(BACK ? i - 1 : i + 1);
    if (DELTA && !(BACK && n == 0)) {
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        const Frag<3> s = split_tiles<3>(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
        for (int mm = 0; mm < IT; mm += 4) {
          Frag<3> f[4];
          f32x4 t[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            f[m] = BACK ? carry_cols<DK>(lds, mm + m, ks) : carry_rows<DK>(lds, mm + m, ks);
            t[m] = x[mm + m];
          }
          mma_tiles(t, f, s);
#pragma unroll
          for (int m = 0; m < 4; ++m) x[mm + m] = t[m];
        }
      }
#pragma unroll
      for (int m = 0; m < IT; ++m) S[m] = x[m];
    }
    keep_chunk_state(start + unit(BACK ? i - 1 : i + 1) * size, col0, S);
  }
}

template <int DK, bool DELTA, bool BACK>
hipError_t join(const ScanArgs& a, hipStream_t stream) {
  constexpr size_t lds = DELTA ? 3 * kCarryPlane<DK> : 16;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(join_kernel<DK, DELTA, BACK>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((join_kernel<DK, DELTA, BACK>),
                     dim3((unsigned)((size_t)a.n_seq * a.heads * (a.d_v / 64))), dim3(256), lds, stream, a);
  return hipGetLastError();
}
template <int DK>
hipError_t join_rule(const ScanArgs& a, bool backward, hipStream_t stream) {
  if (a.rule == kMAMBA2) return backward ? join<DK, false, true>(a, stream) : join<DK, false, false>(a, stream);
  return backward ? join<DK, true, true>(a, stream) : join<DK, true, false>(a, stream);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_join(const ScanArgs& a, bool backward, hipStream_t stream) {
  return a.d_k == 128 ? scan::join_rule<128>(a, backward, stream) : scan::join_rule<64>(a, backward, stream);
}

}  // namespace seed
