// The gradients inside each chunk, for every (chunk, head) at once, from the
// states S and H on both sides of the chunk and E and Y (formulas in
// seed_scan.h).  A gate's gradient is summed over the pairs s < t <= r that
// its decay lies between, each without the gate itself (the decays before
// and behind it), so no quotient is taken and a gate of 0 has its gradient.
#include "seed_scan.h"

namespace seed {
namespace scan {
namespace {

constexpr int kLd = kC + 1;

__device__ __forceinline__ float sum16(float x) {
  x += __shfl_xor(x, 1);
  x += __shfl_xor(x, 2);
  x += __shfl_xor(x, 4);
  x += __shfl_xor(x, 8);
  return x;
}
__device__ __forceinline__ float sum64(float x) {
  x = sum16(x);
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

// Rows of an LDS matrix [64][65] (or of its transpose) as a fragment.
__device__ __forceinline__ void lds_rows(const float* mat, int mt, int ks, bool transposed,
                                         float (&x)[8]) {
  const int row = 16 * mt + (lane_id() & 15), g = lane_id() >> 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = 32 * ks + 16 * (j >> 2) + 4 * g + (j & 3);
    x[j] = transposed ? mat[c * kLd + row] : mat[row * kLd + c];
  }
}

template <int RULE, int DK, int DV, typename T>
__global__ __launch_bounds__(256) void grads_kernel(ScanArgs a) {
  constexpr bool KDA = RULE == kKDA, DELTA = RULE != kMAMBA2;
  constexpr int NT = sizeof(T) == 2 ? 1 : 3;   // terms of an input
  constexpr int NE = DELTA ? 3 : NT;           // terms of u
  extern __shared__ float lds[];
  float* G = lds;                    // [64][65] decays (scalar gates)
  float* dL = G + (KDA ? 0 : kC * kLd);
  float* dM = dL + kC * kLd;
  float* W = dM + kC * kLd;          // gradients of the decays (scalar gates)
  float* dP = W + (KDA ? 0 : kC * kLd);   // [64]
  float* dF = dP + kC;
  float* red = dF + kC;              // [4][64]
  float* hs = red + 4 * kC;          // [DK]
  const Chunk ch = chunk_of_slot(a, blockIdx.x);
  if (ch.n == 0) return;
  const int head = blockIdx.y, tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int l16 = l & 15, g16 = l >> 4, n = ch.n;
  const size_t unit = (size_t)blockIdx.x * a.heads + head;
  const int hk = head / (a.heads / a.key_heads);
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * DV;
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* V = static_cast<const T*>(a.v) + ((size_t)ch.tok * a.heads + head) * DV;
  const T* dO = static_cast<const T*>(a.dO) + ((size_t)ch.tok * a.heads + head) * DV;
  const float* P = reinterpret_cast<const float*>(a.ws + a.at.p) + unit * kC * (KDA ? DK : 1);
  const float* F = reinterpret_cast<const float*>(a.ws + a.at.f) + unit * kC * (KDA ? DK : 1);
  const float* Sc = reinterpret_cast<const float*>(a.ws + a.at.state) + unit * DK * DV;
  const float* Hc = reinterpret_cast<const float*>(a.ws + a.at.grad) + unit * DK * DV;
  const float* E = reinterpret_cast<const float*>(a.ws + a.at.e) + unit * kC * DV;
  const float* Y = reinterpret_cast<const float*>(a.ws + a.at.y) + unit * kC * DV;
  const size_t gate = ((size_t)ch.tok + l) * a.heads + head;
  const float bl = DELTA && l < n ? a.beta[gate] : 0.f;   // lane t: beta_t

  if (!KDA && w == 0) {
    const float gl = l < n ? a.g[gate] : 1.f;
    float cur = 1.f;
    for (int t = 0; t < kC; ++t) {
      const float gt = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gl), t));
      cur = t > l ? cur * gt : 1.f;
      G[t * kLd + l] = t >= l ? cur : 0.f;
    }
  }
  // <H, S>, whole or by key channel
  {
    float all = 0.f;
    for (int i = w; i < DK; i += 4) {
      float x = 0.f;
      for (int j = l; j < DV; j += 64) x += Sc[(size_t)i * DV + j] * Hc[(size_t)i * DV + j];
      if (KDA) {
        x = sum64(x);
        if (l == 0) hs[i] = x;
      } else {
        all += x;
      }
    }
    if (!KDA) {
      all = sum64(all);
      if (l == 0) hs[w] = all;
    }
  }
  // dbeta = Y . E
  if (DELTA) {
    for (int t = 16 * w; t < 16 * w + 16; ++t) {
      float x = 0.f;
      for (int j = l; j < DV; j += 64) x += Y[(size_t)t * DV + j] * E[(size_t)t * DV + j];
      x = sum64(x);
      if (l == 0 && t < n) a.dbeta[((size_t)ch.tok + t) * a.heads + head] = x;
    }
  }
  __syncthreads();

  // a fragment of rows of u, dR and dO (the contracted index along d_v)
  auto rows_u = [&](int tile, int ks) {
    const int t = 16 * tile + l16;
    float x[8];
    if (DELTA) {
      load_row8(E + (size_t)t * DV, 32 * ks, true, x);
      const float b = __shfl(bl, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= b;
    } else {
      load_row8(V + (size_t)t * vld, 32 * ks, t < n, x);
    }
    return split<NE>(x);
  };
  auto rows_dr = [&](int tile, int ks) {
    const int t = 16 * tile + l16;
    float x[8];
    load_row8(Y + (size_t)t * DV, 32 * ks, true, x);
    const float b = __shfl(bl, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= b;
    return split<3>(x);
  };
  auto rows_do = [&](int tile, int ks) {
    const int t = 16 * tile + l16;
    float x[8];
    load_row8(dO + (size_t)t * vld, 32 * ks, t < n, x);
    return split<NT>(x);
  };
  auto rows_in = [&](const T* base, int tile, int ks) {
    const int t = 16 * tile + l16;
    float x[8];
    load_row8(base + (size_t)t * kld, 32 * ks, t < n, x);
    return split<NT>(x);
  };

  // the pairs (t, s): dL, dM, and the gradient of their decay
  for (int sb = 0; sb < 4; ++sb) {
    f32x4 cl = {0.f, 0.f, 0.f, 0.f}, cm = cl, kk = cl, qk = cl;
    if (sb <= w) {
#pragma unroll
      for (int ks = 0; ks < DV / 32; ++ks) {
        const Frag<NE> u = rows_u(sb, ks);
        mma(cm, rows_do(w, ks), u);
        if (DELTA) mma(cl, rows_dr(w, ks), u);
      }
      if (!KDA) {
#pragma unroll
        for (int ks = 0; ks < DK / 32; ++ks) {
          const Frag<NT> k = rows_in(K, sb, ks);
          if (DELTA) mma(kk, rows_in(K, w, ks), k);
          mma(qk, rows_in(Q, w, ks), k);
        }
      }
    }
    const int s = 16 * sb + l16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * g16 + r;
      const float x = s < t ? -cl[r] : 0.f, y = s <= t ? cm[r] : 0.f;
      if (KDA) {
        dL[t * kLd + s] = x;
        dM[t * kLd + s] = y;
      } else {
        dL[t * kLd + s] = x * G[t * kLd + s];
        dM[t * kLd + s] = y * G[t * kLd + s];
        W[t * kLd + s] = s < t ? x * kk[r] + y * qk[r] : 0.f;
      }
    }
  }
  __syncthreads();

  const bool shared = a.key_heads != a.heads;
  float* wq = reinterpret_cast<float*>(a.ws + a.at.dq) + ((size_t)ch.tok * a.heads + head) * DK;
  float* wk = reinterpret_cast<float*>(a.ws + a.at.dk) + ((size_t)ch.tok * a.heads + head) * DK;
  T* oq = static_cast<T*>(a.dq) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  T* ok = static_cast<T*>(a.dk) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  float* tp = reinterpret_cast<float*>(a.ws + a.at.tp) + unit * kC * DK;
  float* tf = reinterpret_cast<float*>(a.ws + a.at.tf) + unit * kC * DK;

  // dQ and dK: the parts through the states, and (scalar gates) the pairs
  float dp[4] = {0.f, 0.f, 0.f, 0.f}, df[4] = {0.f, 0.f, 0.f, 0.f};
  for (int it = 0; it < DK / 16; ++it) {
    const int i = 16 * it + l16;
    f32x4 x1 = {0.f, 0.f, 0.f, 0.f}, x2 = x1, x3 = x1;
#pragma unroll
    for (int ks = 0; ks < DV / 32; ++ks) {
      float x[8];
      load_row8(Sc + (size_t)i * DV, 32 * ks, true, x);
      const Frag<3> s = split<3>(x);
      mma(x1, rows_do(w, ks), s);
      if (DELTA) mma(x2, rows_dr(w, ks), s);
      load_row8(Hc + (size_t)i * DV, 32 * ks, true, x);
      mma(x3, rows_u(w, ks), split<3>(x));
    }
    f32x4 dq, dk;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * g16 + r;
      const float q = t < n ? load_scalar(Q + (size_t)t * kld + i) : 0.f;
      const float k = t < n ? load_scalar(K + (size_t)t * kld + i) : 0.f;
      const float p = KDA ? P[t * DK + i] : P[t], f = KDA ? F[t * DK + i] : F[t];
      dq[r] = p * x1[r];
      dk[r] = f * x3[r] - p * x2[r];
      if (KDA) {
        tp[t * DK + i] = q * x1[r] - k * x2[r];
        tf[t * DK + i] = k * x3[r];
      } else {
        dp[r] += q * x1[r] - k * x2[r];
        df[r] += k * x3[r];
      }
    }
    if (!KDA) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        float kc[8], qc[8], x[8], y[8];
        load_col8(K + i, kld, 32 * ks, n, kc);
        load_col8(Q + i, kld, 32 * ks, n, qc);
        const Frag<NT> kf = split<NT>(kc);
        lds_rows(dM, w, ks, false, x);
        mma(dq, split<3>(x), kf);
        lds_rows(dM, w, ks, true, x);
        mma(dk, split<3>(x), split<NT>(qc));
        if (DELTA) {
          lds_rows(dL, w, ks, false, x);
          lds_rows(dL, w, ks, true, y);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] += y[j];
          mma(dk, split<3>(x), kf);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * g16 + r;
      if (t >= n) continue;
      if (KDA || shared) {
        wq[(size_t)t * a.heads * DK + i] = dq[r];
        wk[(size_t)t * a.heads * DK + i] = dk[r];
      } else {
        store_scalar(oq + (size_t)t * kld + i, dq[r]);
        store_scalar(ok + (size_t)t * kld + i, dk[r]);
      }
    }
  }

  if (!KDA) {
    // dg_t = sum over r >= t > s of G_rt W_rs G_{t-1,s}; s = -1 is the state
    // before the chunk (W = dP, G_{t-1,-1} = P_{t-1}), r = 64 the one behind
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = sum16(dp[r]), y = sum16(df[r]);
      if (l16 == 0) {
        dP[16 * w + 4 * g16 + r] = x;
        dF[16 * w + 4 * g16 + r] = y;
      }
    }
    __syncthreads();
    const int t = l;
    const float before = t == 0 ? 1.f : P[t - 1];
    float acc[17];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = dP[16 * w + j] * before;
    acc[16] = (hs[0] + hs[1] + hs[2] + hs[3]) * before;
    for (int s = 0; s < kC; ++s) {
      const float x = s < t ? G[(t - 1) * kLd + s] : 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[j] += W[(16 * w + j) * kLd + s] * x;
      acc[16] += dF[s] * x;
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) sum += G[(16 * w + j) * kLd + t] * acc[j];
    if (w == 3) sum += F[t] * acc[16];
    red[w * kC + t] = sum;
    __syncthreads();
    if (w == 0 && t < n)
      a.dg[gate] = (red[t] + red[kC + t]) + (red[2 * kC + t] + red[3 * kC + t]);
    return;
  }

  // Gates per key channel: a thread owns a channel and sums pair by pair,
  // its group every NG-th column s.
  if constexpr (KDA) {
    constexpr int NG = 256 / DK;
    float* qs = red + 4 * kC + DK;     // [64][DK]
    float* ks_ = qs + kC * DK;
    float* gs = ks_ + kC * DK;
    const float* gg = a.g + ((size_t)ch.tok * a.heads + head) * DK;
    for (int e = tid; e < kC * DK; e += 256) {
      const int t = e / DK, i = e % DK;
      const bool live = t < n;
      gs[e] = live ? gg[(size_t)t * a.heads * DK + i] : 1.f;
      ks_[e] = live ? load_scalar(K + (size_t)t * kld + i) : 0.f;
      qs[e] = live ? load_scalar(Q + (size_t)t * kld + i) : 0.f;
    }
    __syncthreads();
    const int i = tid % DK, grp = tid / DK;
    float aq[kC], ak[kC], ag[kC];
#pragma unroll
    for (int t = 0; t < kC; ++t) aq[t] = ak[t] = ag[t] = 0.f;
    for (int s = grp; s < n; s += NG) {
      const float k0 = ks_[s * DK + i];
      float dks = 0.f, cur = 0.f, G1[kC];
#pragma unroll
      for (int r = 0; r < kC; ++r) {
        G1[r] = cur;                       // the decay after s through r - 1
        cur = r > s ? cur * gs[r * DK + i] : (r == s ? 1.f : 0.f);
        const float m = dM[r * kLd + s] * cur, x = dL[r * kLd + s] * cur;
        aq[r] += m * k0;
        ak[r] += x * k0;
        dks += m * qs[r * DK + i] + x * ks_[r * DK + i];
      }
      float c = 0.f, after = 1.f;
#pragma unroll
      for (int r = kC - 1; r >= 0; --r) {
        const float g = gs[r * DK + i];
        if (r > s) {
          c = c * after + k0 * (dL[r * kLd + s] * ks_[r * DK + i] + dM[r * kLd + s] * qs[r * DK + i]);
          ag[r] += G1[r] * c;
        }
        after = g;
        if (r == s) ak[r] += dks;
      }
    }
    if (grp == 0) {
      float c = hs[i], after = 1.f;
#pragma unroll
      for (int t = kC - 1; t >= 0; --t) {
        c = c * after + tp[t * DK + i];
        after = gs[t * DK + i];
        ag[t] += (t == 0 ? 1.f : P[(t - 1) * DK + i]) * c;
      }
      float b = 0.f;
#pragma unroll
      for (int t = 0; t < kC; ++t) {
        ag[t] += F[t * DK + i] * b;
        b = b * gs[t * DK + i] + tf[t * DK + i];
      }
    }
    __syncthreads();   // q, k and g are used up: their places take the sums
    for (int turn = 0; turn < NG; ++turn) {
      if (grp == turn) {
#pragma unroll
        for (int t = 0; t < kC; ++t) {
          const int e = t * DK + i;
          qs[e] = aq[t] + (turn ? qs[e] : 0.f);
          ks_[e] = ak[t] + (turn ? ks_[e] : 0.f);
          gs[e] = ag[t] + (turn ? gs[e] : 0.f);
        }
      }
      __syncthreads();
    }
    for (int e = tid; e < n * DK; e += 256) {
      const int t = e / DK, c = e % DK;
      const size_t at = (size_t)t * a.heads * DK + c;
      const float q = wq[at] + qs[e], k = wk[at] + ks_[e];
      if (shared) {
        wq[at] = q;
        wk[at] = k;
      } else {
        store_scalar(oq + (size_t)t * kld + c, q);
        store_scalar(ok + (size_t)t * kld + c, k);
      }
      a.dg[((size_t)ch.tok * a.heads + head) * DK + at] = gs[e];
    }
  }
}

// Gradients of keys and queries that several heads share: the sum over the
// group in head order.  Rows outside every sequence are left as they were.
template <typename T>
__global__ __launch_bounds__(256) void share_kernel(ScanArgs a) {
  const int per = a.heads / a.key_heads;
  const size_t total = (size_t)a.tokens * a.key_heads * a.d_k;
  const int last = a.cu ? min(max(a.cu[a.n_seq], 0), a.tokens) : a.tokens;
  const int first = a.cu ? min(max(a.cu[0], 0), last) : 0;
  for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (size_t)gridDim.x * 256) {
    const int i = (int)(e % a.d_k);
    const size_t th = e / a.d_k;
    const size_t tok = th / a.key_heads;
    if (tok < (size_t)first || tok >= (size_t)last) continue;
    const size_t at = (tok * a.heads + (th % a.key_heads) * per) * a.d_k + i;
    const float* wq = reinterpret_cast<const float*>(a.ws + a.at.dq);
    const float* wk = reinterpret_cast<const float*>(a.ws + a.at.dk);
    float q = 0.f, k = 0.f;
    for (int h = 0; h < per; ++h) {
      q += wq[at + (size_t)h * a.d_k];
      k += wk[at + (size_t)h * a.d_k];
    }
    store_scalar(static_cast<T*>(a.dq) + e, q);
    store_scalar(static_cast<T*>(a.dk) + e, k);
  }
}

template <int RULE, int DK, int DV, typename T>
hipError_t grads(const ScanArgs& a, hipStream_t stream) {
  constexpr bool KDA = RULE == kKDA;
  const size_t lds = ((KDA ? 2 : 4) * kC * kLd + 6 * kC + DK + (KDA ? 3 * kC * DK : 0)) * sizeof(float);
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(grads_kernel<RULE, DK, DV, T>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((grads_kernel<RULE, DK, DV, T>), dim3(a.slots, a.heads), dim3(256), lds, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess || a.key_heads == a.heads) return e;
  const size_t total = (size_t)a.tokens * a.key_heads * DK;
  const size_t blocks = (total + 255) / 256;
  hipLaunchKernelGGL((share_kernel<T>), dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256),
                     0, stream, a);
  return hipGetLastError();
}
template <int DK, int DV, typename T>
hipError_t grads_rule(const ScanArgs& a, hipStream_t stream) {
  switch (a.rule) {
    case kGDN: return grads<kGDN, DK, DV, T>(a, stream);
    case kKDA: return grads<kKDA, DK, DV, T>(a, stream);
    default: return grads<kMAMBA2, DK, DV, T>(a, stream);
  }
}
template <typename T>
hipError_t grads_shape(const ScanArgs& a, hipStream_t stream) {
  if (a.d_k == 128)
    return a.d_v == 128 ? grads_rule<128, 128, T>(a, stream) : grads_rule<128, 64, T>(a, stream);
  return grads_rule<64, 64, T>(a, stream);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_grads(const ScanArgs& a, hipStream_t stream) {
  return a.bf16 ? scan::grads_shape<bf16_t>(a, stream) : scan::grads_shape<float>(a, stream);
}

}  // namespace seed
