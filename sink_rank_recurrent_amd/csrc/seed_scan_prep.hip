// Inside each chunk of the recurrence: the decays and the triangles N and M
// (formulas in seed_scan.h), for every (chunk, head) at once.
#include "seed_scan.h"

namespace seed {
namespace scan {
namespace {


// A 16 x 16 x 16 product in fp32: a's rows from LDS, b an accumulator tile.
__device__ __forceinline__ void mma_f32(f32x4& c, const f32x4& a, const f32x4& b) {
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
}

// N = (I + L beta)^-1 L in place of L [64][kRow], by blocks of 16:
//   N_ic = X_ii (L_ic - sum over c <= j < i of L_ij beta_j N_jc),
// X_ii = (I + L_ii beta_i)^-1 by substitution.  Wave w inverts block w, then
// takes column w of blocks, its tiles staying in registers as the next
// product's right operand.  X: [4][16][20].
__device__ __forceinline__ void solve(float* L, float* X, const float* beta, int w) {
  const int l = lane_id(), l16 = l & 15, g = l >> 4;
  if (l < 16) {   // lane c: column c of X_ww
    float x[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      float v = t == l ? 1.f : 0.f;
#pragma unroll
      for (int s = 0; s < t; ++s) v -= L[(16 * w + t) * kRow + 16 * w + s] * x[s];
      X[(w * 16 + t) * 20 + l] = v;
      x[t] = v * beta[16 * w + t];
    }
  }
  __syncthreads();
  f32x4 N[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    N[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (i < w) continue;
    f32x4 acc;
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = L[(16 * i + 4 * g + r) * kRow + 16 * w + l16];
#pragma unroll
    for (int j = 0; j < i; ++j) {
      if (j < w) continue;
      const f32x4 a = *reinterpret_cast<const f32x4*>(L + (16 * i + l16) * kRow + 16 * j + 4 * g);
      const f32x4 b = *reinterpret_cast<const f32x4*>(beta + 16 * j + 4 * g);
      mma_f32(acc, -(a * b), N[j]);
    }
    mma_f32(N[i], *reinterpret_cast<const f32x4*>(X + (i * 16 + l16) * 20 + 4 * g), acc);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) L[(16 * i + 4 * g + r) * kRow + 16 * w + l16] = N[i][r];
  __syncthreads();
}

// The triangle of an LDS matrix as a pack (transposed: of its transpose).
__device__ __forceinline__ void pack_triangle(uint16_t* __restrict__ pack, const float* mat,
                                              bool transposed, int mt, int ks) {
  const int frag = transposed ? upper_frag(mt, ks) : lower_frag(mt, ks);
  if (frag < 0) return;
  const int row = 16 * mt + (lane_id() & 15), g = lane_id() >> 4;
  float x[8];
  if (transposed) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = mat[(32 * ks + 16 * (j >> 2) + 4 * g + (j & 3)) * kRow + row];
  } else {
    tiles_to_floats(*reinterpret_cast<const f32x4*>(mat + row * kRow + 32 * ks + 4 * g),
                    *reinterpret_cast<const f32x4*>(mat + row * kRow + 32 * ks + 16 + 4 * g), x);
  }
  store_pack(pack, frag, split<3>(x));
}

// Half a fragment (slots 4 h .. 4 h + 3): one accumulator tile of the
// transposed product.
__device__ __forceinline__ void store_half(uint16_t* __restrict__ pack, int frag, int h,
                                           const f32x4& c) {
  const float x[8] = {c[0], c[1], c[2], c[3], 0.f, 0.f, 0.f, 0.f};
  const Frag<3> f = split<3>(x);
#pragma unroll
  for (int n = 0; n < 3; ++n)
    *reinterpret_cast<uint2*>(pack + (size_t)(frag * 3 + n) * kFrag + lane_id() * 8 + 4 * h) =
        make_uint2(f.t[n][0], f.t[n][1]);
}

// Four waves a (chunk, head); wave a has the tokens 16 a .. + 15 as rows.
template <int RULE, int DK, typename T, bool BWD>
__global__ __launch_bounds__(256) void prep_scalar_kernel(ScanArgs a) {
  constexpr int NT = sizeof(T) == 2 ? 1 : 3;
  constexpr bool DELTA = RULE != kMAMBA2;
  __shared__ __attribute__((aligned(16))) float L[DELTA ? kC * kRow : 4];
  __shared__ __attribute__((aligned(16))) float X[DELTA ? 64 * 20 : 4];
  __shared__ __attribute__((aligned(16))) float bt[kC];
  __shared__ __attribute__((aligned(16))) uint16_t kl[4 * (DK / 32) * NT * kFrag];   // K's fragments
  __shared__ Decay dec;
  const Chunk ch = chunk_of_slot(a, blockIdx.x);
  if (ch.n == 0) return;
  const int head = blockIdx.y, w = threadIdx.x >> 6, l = lane_id(), g16 = l >> 4, l16 = l & 15;
  const size_t unit = (size_t)blockIdx.x * a.heads + head;
  const int hk = head / (a.heads / a.key_heads);
  const size_t ld = (size_t)a.key_heads * DK;
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  uint16_t* mp = reinterpret_cast<uint16_t*>(a.ws + a.at.m_pack) + unit * (kTriFrags * 3 * kFrag);

  // the wave's rows of K and Q
  const int t0 = 16 * w + l16;
  Frag<NT> kt[DK / 32], qt[DK / 32];
#pragma unroll
  for (int ks = 0; ks < DK / 32; ++ks) {
    float x[8];
    load_piece(K + (size_t)t0 * ld, 32 * ks, t0 < ch.n, x);
    kt[ks] = split<NT>(x);
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<u32x4*>(kl + (((w * (DK / 32) + ks) * NT + n) * 64 + l) * 8) = kt[ks].t[n];
    load_piece(Q + (size_t)t0 * ld, 32 * ks, t0 < ch.n, x);
    qt[ks] = split<NT>(x);
  }
  if (w == 0) {
    const size_t gate = ((size_t)ch.tok + l) * a.heads + head;
    float P, F;
    decays(dec, l < ch.n ? a.g[gate] : 1.f, P, F);
    reinterpret_cast<float*>(a.ws + a.at.p)[unit * kC + l] = P;
    reinterpret_cast<float*>(a.ws + a.at.f)[unit * kC + l] = F;
    if (DELTA) {
      bt[l] = l < ch.n ? a.beta[gate] : 0.f;
      reinterpret_cast<float*>(a.ws + a.at.b)[unit * kC + l] = bt[l];
    }
  }
  __syncthreads();

  for (int b = 0; b < 4; ++b) {
    // lane (t, s): its row of the right operand and four rows of the left;
    // backward the left operand is Q, and M's tile comes out transposed
    f32x4 ll = {0.f, 0.f, 0.f, 0.f}, mm = ll;
    if (b <= w) {
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        Frag<NT> kb;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          kb.t[n] = *reinterpret_cast<const u32x4*>(kl + (((b * (DK / 32) + ks) * NT + n) * 64 + l) * 8);
        if (DELTA) mma(ll, kb, kt[ks]);
        if (BWD) mma(mm, qt[ks], kb);
        else mma(mm, kb, qt[ks]);
      }
    }
    f32x4 gl = {0.f, 0.f, 0.f, 0.f}, gm = gl;
    const int t = 16 * w + l16, s = 16 * b + 4 * g16;        // L, and M forward
    const int tm = 16 * w + 4 * g16, sm = 16 * b + l16;      // M backward
    if (b < w) {
      const float mid = dec.mid[4 * w + b];
      gl = *reinterpret_cast<const f32x4*>(dec.suf + s) * (dec.pre[t] * mid);
      gm = BWD ? *reinterpret_cast<const f32x4*>(dec.pre + tm) * (dec.suf[sm] * mid) : gl;
    } else if (b == w) {
      gl = inside<false>(dec.gate, t, s);
      gm = BWD ? inside<true>(dec.gate, tm, sm) : gl;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        gm[r] = (BWD ? sm <= tm + r : s + r <= t) ? gm[r] : 0.f;
        gl[r] = s + r < t ? gl[r] : 0.f;
      }
    }
    if (DELTA) *reinterpret_cast<f32x4*>(L + (16 * w + l16) * kRow + 16 * b + 4 * g16) = ll * gl;
    mm *= gm;
    if (BWD) {
      // rows s of tile b, tokens of tile w; a block's zero half is written too
      if (upper_frag(b, w >> 1) >= 0) store_half(mp, upper_frag(b, w >> 1), w & 1, mm);
    } else {
      if (lower_frag(w, b >> 1) >= 0) store_half(mp, lower_frag(w, b >> 1), b & 1, mm);
    }
  }
  if (DELTA) {
    __syncthreads();
    solve(L, X, bt, w);
    uint16_t* np = reinterpret_cast<uint16_t*>(a.ws + a.at.n_pack) + unit * (kTriFrags * 3 * kFrag);
    for (int i = w; i < 8; i += 4) pack_triangle(np, L, false, i >> 1, i & 1);
    if (BWD) {
      uint16_t* tp =
          reinterpret_cast<uint16_t*>(a.ws + a.at.nt_pack) + unit * (kTriFrags * 3 * kFrag);
      for (int i = w; i < 8; i += 4) pack_triangle(tp, L, true, i >> 1, i & 1);
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
  float* Lm = qq + ((kC * LR + 3) & ~3);   // [64][kRow]
  float* Mm = Lm + kC * kRow;
  float* bt = Mm + kC * kRow;
  float* X = bt + kC;                      // [4][16][20]
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
        Lm[t * kRow + l] = turn == 0 ? x : Lm[t * kRow + l] + x;
        Mm[t * kRow + l] = turn == 0 ? y : Mm[t * kRow + l] + y;
      }
    }
    __syncthreads();
  }
  solve(Lm, X, bt, w);
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
    const size_t lds = (3 * kC * (DK + 1) + 2 * kC * kRow + kC + 64 * 20) * sizeof(float);
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(prep_kda_kernel<DK, T, BWD>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((prep_kda_kernel<DK, T, BWD>), grid, dim3(256), lds, stream, a);
  } else if (a.rule == kGDN) {
    hipLaunchKernelGGL((prep_scalar_kernel<kGDN, DK, T, BWD>), grid, dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL((prep_scalar_kernel<kMAMBA2, DK, T, BWD>), grid, dim3(256), 0, stream, a);
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
