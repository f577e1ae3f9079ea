// Inside each chunk of the recurrence: the decays and the triangles N and M
// (formulas in seed_scan.h), for every (chunk, head) at once.
#include "seed_scan.h"

namespace seed {
namespace scan {
namespace {

constexpr int kLd = kC + 1;   // LDS rows, padded against bank conflicts

// N = (I + L beta)^-1 L in place of L: row t is L_t - sum_{s<t} L_ts beta_s N_s.
// Lane c holds column c of beta N; one wave.
__device__ __forceinline__ void solve(float* Lm, const float* beta) {
  const int c = lane_id();
  float m[kC];
#pragma unroll
  for (int t = 0; t < kC; ++t) {
    float x = Lm[t * kLd + c];
#pragma unroll
    for (int s = 0; s < t; ++s) x -= Lm[t * kLd + s] * m[s];
    m[t] = beta[t] * x;
    Lm[t * kLd + c] = x;
  }
}

// The triangle of an LDS matrix as a pack (upper: of its transpose).
__device__ __forceinline__ void pack_triangle(uint16_t* __restrict__ pack, const float* mat,
                                              bool transposed, int mt, int ks) {
  const int frag = transposed ? upper_frag(mt, ks) : lower_frag(mt, ks);
  if (frag < 0) return;
  const int row = 16 * mt + (lane_id() & 15), g = lane_id() >> 4;
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int col = 32 * ks + 16 * (j >> 2) + 4 * g + (j & 3);
    x[j] = transposed ? mat[col * kLd + row] : mat[row * kLd + col];
  }
  store_pack(pack, frag, split<3>(x));
}

// One 16 x 16 tile A B^T of rows of two row-major arrays, DK long.
template <int DK, int NT, typename T>
__device__ __forceinline__ f32x4 row_product(const T* __restrict__ a, const T* __restrict__ b,
                                             size_t ld, int ta, int tb, int n) {
  const int r = lane_id() & 15;
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < DK / 32; ++ks) {
    float x[8], y[8];
    load_row8(a + (size_t)(16 * ta + r) * ld, 32 * ks, 16 * ta + r < n, x);
    load_row8(b + (size_t)(16 * tb + r) * ld, 32 * ks, 16 * tb + r < n, y);
    mma(c, split<NT>(x), split<NT>(y));
  }
  return c;
}

template <int RULE, int DK, typename T, bool BWD>
__global__ __launch_bounds__(64) void prep_scalar_kernel(ScanArgs a) {
  constexpr int NT = sizeof(T) == 2 ? 1 : 3;
  __shared__ float G[kC * kLd];
  __shared__ float Lm[kC * kLd];
  __shared__ float bt[kC];
  const Chunk ch = chunk_of_slot(a, blockIdx.x);
  if (ch.n == 0) return;
  const int head = blockIdx.y, l = threadIdx.x, g16 = l >> 4, l16 = l & 15;
  const size_t unit = (size_t)blockIdx.x * a.heads + head;
  const int hk = head / (a.heads / a.key_heads);
  const size_t ld = (size_t)a.key_heads * DK;
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const size_t gate = ((size_t)ch.tok + l) * a.heads + head;

  // the decays: lane s multiplies its own column G_.s downwards
  const float gl = l < ch.n ? a.g[gate] : 1.f;
  float cur = 1.f, p = 1.f;
  for (int t = 0; t < kC; ++t) {
    const float gt = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gl), t));
    cur = t > l ? cur * gt : 1.f;
    p = t <= l ? p * gt : p;
    G[t * kLd + l] = t >= l ? cur : 0.f;
  }
  reinterpret_cast<float*>(a.ws + a.at.p)[unit * kC + l] = p;
  reinterpret_cast<float*>(a.ws + a.at.f)[unit * kC + l] = cur;
  if (RULE != kMAMBA2) {
    bt[l] = l < ch.n ? a.beta[gate] : 0.f;
    reinterpret_cast<float*>(a.ws + a.at.b)[unit * kC + l] = bt[l];
  }
  __syncthreads();

  if (RULE != kMAMBA2) {
    for (int ta = 0; ta < 4; ++ta) {
      for (int tb = 0; tb < 4; ++tb) {
        const int t = 16 * ta + l16;
        f32x4 c = {0.f, 0.f, 0.f, 0.f};
        if (tb <= ta) c = row_product<DK, NT>(K, K, ld, tb, ta, ch.n);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int s = 16 * tb + 4 * g16 + r;
          Lm[t * kLd + s] = s < t ? c[r] * G[t * kLd + s] : 0.f;
        }
      }
    }
    __syncthreads();
    solve(Lm, bt);
    __syncthreads();
    uint16_t* np = reinterpret_cast<uint16_t*>(a.ws + a.at.n_pack) + unit * (kTriFrags * 3 * kFrag);
    for (int i = 0; i < 8; ++i) pack_triangle(np, Lm, false, i >> 1, i & 1);
    if (BWD) {
      uint16_t* tp =
          reinterpret_cast<uint16_t*>(a.ws + a.at.nt_pack) + unit * (kTriFrags * 3 * kFrag);
      for (int i = 0; i < 8; ++i) pack_triangle(tp, Lm, true, i >> 1, i & 1);
    }
    __syncthreads();
  }

  // M (or M^T), already in fragment order as the product K Q^T (Q K^T)
  uint16_t* mp = reinterpret_cast<uint16_t*>(a.ws + a.at.m_pack) + unit * (kTriFrags * 3 * kFrag);
  for (int mt = 0; mt < 4; ++mt) {
    for (int ks = 0; ks < 2; ++ks) {
      const int frag = BWD ? upper_frag(mt, ks) : lower_frag(mt, ks);
      if (frag < 0) continue;
      float x[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kt = 2 * ks + h;
        f32x4 c = {0.f, 0.f, 0.f, 0.f};
        if (BWD ? kt >= mt : kt <= mt)
          c = BWD ? row_product<DK, NT>(Q, K, ld, kt, mt, ch.n)
                  : row_product<DK, NT>(K, Q, ld, kt, mt, ch.n);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * mt + l16, col = 16 * kt + 4 * g16 + r;
          x[4 * h + r] = c[r] * (BWD ? G[col * kLd + row] : G[row * kLd + col]);
        }
      }
      store_pack(mp, frag, split<3>(x));
    }
  }
}

// Gates per key channel: every pair's decay differs by channel, so the
// triangles are summed pair by pair, lane s running down column s.  A wave
// takes a quarter of the channels.
template <int DK, typename T, bool BWD>
__global__ __launch_bounds__(256) void prep_kda_kernel(ScanArgs a) {
  constexpr int LR = DK + 1;
  extern __shared__ float lds[];
  float* gs = lds;                 // [64][DK + 1]
  float* kk = gs + kC * LR;
  float* qq = kk + kC * LR;
  float* Lm = qq + kC * LR;        // [64][65]
  float* Mm = Lm + kC * kLd;
  float* bt = Mm + kC * kLd;
  const Chunk ch = chunk_of_slot(a, blockIdx.x);
  if (ch.n == 0) return;
  const int head = blockIdx.y, tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const size_t unit = (size_t)blockIdx.x * a.heads + head;
  const int hk = head / (a.heads / a.key_heads);
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const float* gg = a.g + ((size_t)ch.tok * a.heads + head) * DK;

  for (int e = tid; e < kC * DK; e += 256) {
    const int t = e / DK, i = e % DK;
    const bool live = t < ch.n;
    gs[t * LR + i] = live ? gg[(size_t)t * a.heads * DK + i] : 1.f;
    kk[t * LR + i] = live ? load_scalar(K + (size_t)t * a.key_heads * DK + i) : 0.f;
    qq[t * LR + i] = live ? load_scalar(Q + (size_t)t * a.key_heads * DK + i) : 0.f;
  }
  if (tid < kC) {
    bt[tid] = tid < ch.n ? a.beta[((size_t)ch.tok + tid) * a.heads + head] : 0.f;
    reinterpret_cast<float*>(a.ws + a.at.b)[unit * kC + tid] = bt[tid];
  }
  __syncthreads();

  float* P = reinterpret_cast<float*>(a.ws + a.at.p) + unit * kC * DK;
  float* F = reinterpret_cast<float*>(a.ws + a.at.f) + unit * kC * DK;
  if (tid < DK) {
    float x = 1.f;
    for (int t = 0; t < kC; ++t) {
      x *= gs[t * LR + tid];
      P[t * DK + tid] = x;
    }
    x = 1.f;
    for (int t = kC - 1; t >= 0; --t) {
      F[t * DK + tid] = x;
      x *= gs[t * LR + tid];
    }
  }

  float accL[kC], accM[kC];
#pragma unroll
  for (int t = 0; t < kC; ++t) accL[t] = accM[t] = 0.f;
  for (int i = w * (DK / 4); i < (w + 1) * (DK / 4); ++i) {
    const float ks = kk[l * LR + i];
    float cur = 0.f;
#pragma unroll
    for (int t = 0; t < kC; ++t) {
      cur = t > l ? cur * gs[t * LR + i] : (t == l ? ks : 0.f);
      accL[t] += kk[t * LR + i] * cur;
      accM[t] += qq[t * LR + i] * cur;
    }
  }
  for (int turn = 0; turn < 4; ++turn) {
    if (w == turn) {
#pragma unroll
      for (int t = 0; t < kC; ++t) {
        const float x = t > l ? accL[t] : 0.f, y = accM[t];
        Lm[t * kLd + l] = turn == 0 ? x : Lm[t * kLd + l] + x;
        Mm[t * kLd + l] = turn == 0 ? y : Mm[t * kLd + l] + y;
      }
    }
    __syncthreads();
  }
  if (w == 0) solve(Lm, bt);
  __syncthreads();
  uint16_t* np = reinterpret_cast<uint16_t*>(a.ws + a.at.n_pack) + unit * (kTriFrags * 3 * kFrag);
  uint16_t* mp = reinterpret_cast<uint16_t*>(a.ws + a.at.m_pack) + unit * (kTriFrags * 3 * kFrag);
  for (int i = w; i < 8; i += 4) {
    pack_triangle(np, Lm, false, i >> 1, i & 1);
    pack_triangle(mp, Mm, BWD, i >> 1, i & 1);
    if (BWD) {
      uint16_t* tp =
          reinterpret_cast<uint16_t*>(a.ws + a.at.nt_pack) + unit * (kTriFrags * 3 * kFrag);
      pack_triangle(tp, Lm, true, i >> 1, i & 1);
    }
  }
}

template <int DK, typename T, bool BWD>
hipError_t prep(const ScanArgs& a, hipStream_t stream) {
  const dim3 grid(a.slots, a.heads);
  if (a.rule == kKDA) {
    const size_t lds = (3 * kC * (DK + 1) + 2 * kC * kLd + kC) * sizeof(float);
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(prep_kda_kernel<DK, T, BWD>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((prep_kda_kernel<DK, T, BWD>), grid, dim3(256), lds, stream, a);
  } else if (a.rule == kGDN) {
    hipLaunchKernelGGL((prep_scalar_kernel<kGDN, DK, T, BWD>), grid, dim3(64), 0, stream, a);
  } else {
    hipLaunchKernelGGL((prep_scalar_kernel<kMAMBA2, DK, T, BWD>), grid, dim3(64), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_prep(const ScanArgs& a, bool backward, hipStream_t stream) {
  using namespace scan;
  if (a.d_k == 128) {
    if (a.bf16) return backward ? prep<128, bf16_t, true>(a, stream) : prep<128, bf16_t, false>(a, stream);
    return backward ? prep<128, float, true>(a, stream) : prep<128, float, false>(a, stream);
  }
  if (a.bf16) return backward ? prep<64, bf16_t, true>(a, stream) : prep<64, bf16_t, false>(a, stream);
  return backward ? prep<64, float, true>(a, stream) : prep<64, float, false>(a, stream);
}

}  // namespace seed
