// The recurrence from chunk to chunk, and back.  Columns of the state do not
// mix: a wave owns 16 of them and carries them through a sequence's chunks
// in its accumulators; every product's result is the next one's right
// operand in the registers it is already in (seed_scan.h).
#include "seed_scan.h"

namespace seed {
namespace scan {
namespace {

template <int N>
__device__ __forceinline__ Frag<N> split_tiles(const f32x4& a, const f32x4& b) {
  float x[8];
  tiles_to_floats(a, b, x);
  return split<N>(x);
}

// A key or query fragment, its rows times `scale` ([64][DK], KDA) where
// there is one.
template <int NT, bool SCALED, typename T>
__device__ __forceinline__ Frag<NT> key_rows(const T* __restrict__ base, size_t ld,
                                             const float* __restrict__ scale, int DK, int mt,
                                             int ks, int n) {
  const int t = 16 * mt + (lane_id() & 15);
  float x[8];
  load_row8(base + (size_t)t * ld, 32 * ks, t < n, x);
  if (SCALED) {
    float s[8];
    load_row8(scale + (size_t)t * DK, 32 * ks, true, s);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= s[j];
  }
  return split<NT>(x);
}
template <int NT, bool SCALED, typename T>
__device__ __forceinline__ Frag<NT> key_cols(const T* __restrict__ base, size_t ld,
                                             const float* __restrict__ scale, int DK, int it,
                                             int ks, int n) {
  const int i = 16 * it + (lane_id() & 15);
  float x[8];
  load_col8(base + i, ld, 32 * ks, n, x);
  if (SCALED) {
    float s[8];
    load_col8(scale + i, (size_t)DK, 32 * ks, kC, s);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= s[j];
  }
  return split<NT>(x);
}

// A 64-vector of the chunk in the accumulators' row order: rows 16 m + 4 g + r.
__device__ __forceinline__ f32x4 row_vec(const float* __restrict__ p, int m) {
  float x[4];
  load_vec<4>(p + 16 * m + 4 * (lane_id() >> 4), x);
  return f32x4{x[0], x[1], x[2], x[3]};
}

__device__ __forceinline__ f32x4 beta_rows(const ScanArgs& a, const Chunk& ch, int head, int m) {
  f32x4 b;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int t = 16 * m + 4 * (lane_id() >> 4) + r;
    b[r] = t < ch.n ? a.beta[((size_t)ch.tok + t) * a.heads + head] : 0.f;
  }
  return b;
}

// Columns of a [tokens][heads][d_v] array as accumulator tiles.
template <typename T>
__device__ __forceinline__ f32x4 load_tile(const T* __restrict__ p, size_t ld, int m, int n) {
  f32x4 x;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int t = 16 * m + 4 * (lane_id() >> 4) + r;
    x[r] = t < n ? load_scalar(p + (size_t)t * ld) : 0.f;
  }
  return x;
}
template <typename T>
__device__ __forceinline__ void store_tile(T* __restrict__ p, size_t ld, int m, int n,
                                           const f32x4& x) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int t = 16 * m + 4 * (lane_id() >> 4) + r;
    if (t < n) store_scalar(p + (size_t)t * ld, x[r]);
  }
}

// grid: n_seq * heads * (d_v / 64), a wave for 16 columns.  SAVE keeps each
// chunk's incoming state and E for the backward pass and writes no read-outs.
template <int RULE, int DK, typename T, bool SAVE>
__global__ __launch_bounds__(256) void forward_kernel(ScanArgs a) {
  constexpr bool KDA = RULE == kKDA, DELTA = RULE != kMAMBA2;
  constexpr int NT = sizeof(T) == 2 && !KDA ? 1 : 3;
  constexpr int IT = DK / 16;
  const int w = threadIdx.x >> 6, g = lane_id() >> 4;
  const int blocks = a.d_v / 64;
  const int sh = blockIdx.x / blocks, seq = sh / a.heads, head = sh % a.heads;
  const int col = (blockIdx.x % blocks) * 64 + w * 16 + (lane_id() & 15);
  const int hk = head / (a.heads / a.key_heads);
  const Range rg = sequence(a, seq);
  const int chunks = (rg.len + kC - 1) / kC, base = slot_base(rg, seq);
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * a.d_v;
  const size_t state = ((size_t)seq * a.heads + head) * DK * a.d_v + col;

  f32x4 S[IT];
#pragma unroll
  for (int m = 0; m < IT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      S[m][r] = a.S0 ? a.S0[state + (size_t)(16 * m + 4 * g + r) * a.d_v] : 0.f;

  for (int c = 0; c < chunks; ++c) {
    const int tok = rg.start + c * kC, n = min(kC, rg.len - c * kC);
    const Chunk ch{seq, tok, n, c};
    const size_t unit = (size_t)(base + c) * a.heads + head;
    const T* K = static_cast<const T*>(a.k) + ((size_t)tok * a.key_heads + hk) * DK;
    const T* Q = static_cast<const T*>(a.q) + ((size_t)tok * a.key_heads + hk) * DK;
    const T* V = static_cast<const T*>(a.v) + ((size_t)tok * a.heads + head) * a.d_v + col;
    const float* P = reinterpret_cast<const float*>(a.ws + a.at.p) + unit * kC * (KDA ? DK : 1);
    const float* F = reinterpret_cast<const float*>(a.ws + a.at.f) + unit * kC * (KDA ? DK : 1);
    const uint16_t* Np =
        reinterpret_cast<const uint16_t*>(a.ws + a.at.n_pack) + unit * (kTriFrags * 3 * kFrag);
    const uint16_t* Mp =
        reinterpret_cast<const uint16_t*>(a.ws + a.at.m_pack) + unit * (kTriFrags * 3 * kFrag);

    if (SAVE) {
      float* Sc = reinterpret_cast<float*>(a.ws + a.at.state) + unit * DK * a.d_v + col;
#pragma unroll
      for (int m = 0; m < IT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) Sc[(size_t)(16 * m + 4 * g + r) * a.d_v] = S[m][r];
    }

    f32x4 R[4], O[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) R[m] = O[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      const Frag<3> s = split_tiles<3>(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (DELTA) mma(R[m], key_rows<NT, KDA>(K, kld, P, DK, m, ks, n), s);
        if (!SAVE) mma(O[m], key_rows<NT, KDA>(Q, kld, P, DK, m, ks, n), s);
      }
    }
    f32x4 u[4], b[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 v = load_tile(V, vld, m, n);
      f32x4 p = {1.f, 1.f, 1.f, 1.f};
      if (!KDA) p = row_vec(P, m);
      R[m] = v - p * R[m];
      O[m] = p * O[m];
      if (DELTA) b[m] = beta_rows(a, ch, head, m);
    }
    if (DELTA) {
      Frag<3> x[2];
      x[0] = split_tiles<3>(b[0] * R[0], b[1] * R[1]);
      x[1] = split_tiles<3>(b[2] * R[2], b[3] * R[3]);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (lower_frag(m, ks) >= 0) mma(y, load_pack(Np, lower_frag(m, ks)), x[ks]);
        R[m] -= y;
      }
      if (SAVE) {
        float* E = reinterpret_cast<float*>(a.ws + a.at.e) + unit * kC * a.d_v + col;
#pragma unroll
        for (int m = 0; m < 4; ++m) store_tile(E, (size_t)a.d_v, m, kC, R[m]);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) u[m] = b[m] * R[m];
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) u[m] = R[m];
    }
    if (!SAVE) {
      Frag<3> x[2];
      x[0] = split_tiles<3>(u[0], u[1]);
      x[1] = split_tiles<3>(u[2], u[3]);
      T* out = static_cast<T*>(a.o) + ((size_t)tok * a.heads + head) * a.d_v + col;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (lower_frag(m, ks) >= 0) mma(O[m], load_pack(Mp, lower_frag(m, ks)), x[ks]);
        store_tile(out, vld, m, n, O[m]);
      }
    }
    // S' = P_end S + (F K)^T u
    if (!KDA) {
      const float last = P[kC - 1];
#pragma unroll
      for (int m = 0; m < 4; ++m) u[m] *= row_vec(F, m);
#pragma unroll
      for (int m = 0; m < IT; ++m) S[m] *= last;
    } else {
#pragma unroll
      for (int m = 0; m < IT; ++m) S[m] *= row_vec(P + (kC - 1) * DK, m);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Frag<3> x = split_tiles<3>(u[2 * ks], u[2 * ks + 1]);
#pragma unroll
      for (int m = 0; m < IT; ++m) mma(S[m], key_cols<NT, KDA>(K, kld, F, DK, m, ks, n), x);
    }
  }
  if (!SAVE) {
#pragma unroll
    for (int m = 0; m < IT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) a.S[state + (size_t)(16 * m + 4 * g + r) * a.d_v] = S[m][r];
  }
}

// The chunks from the last to the first, H the gradient of the state behind
// the chunk.  Keeps H and (delta rules) Y, writes dV and dS0.
template <int RULE, int DK, typename T>
__global__ __launch_bounds__(256) void reverse_kernel(ScanArgs a) {
  constexpr bool KDA = RULE == kKDA, DELTA = RULE != kMAMBA2;
  constexpr int NT = sizeof(T) == 2 && !KDA ? 1 : 3;
  constexpr int NV = sizeof(T) == 2 ? 1 : 3;
  constexpr int IT = DK / 16;
  const int w = threadIdx.x >> 6, g = lane_id() >> 4;
  const int blocks = a.d_v / 64;
  const int sh = blockIdx.x / blocks, seq = sh / a.heads, head = sh % a.heads;
  const int col = (blockIdx.x % blocks) * 64 + w * 16 + (lane_id() & 15);
  const int hk = head / (a.heads / a.key_heads);
  const Range rg = sequence(a, seq);
  const int chunks = (rg.len + kC - 1) / kC, base = slot_base(rg, seq);
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * a.d_v;
  const size_t state = ((size_t)seq * a.heads + head) * DK * a.d_v + col;

  f32x4 H[IT];
#pragma unroll
  for (int m = 0; m < IT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      H[m][r] = a.dS ? a.dS[state + (size_t)(16 * m + 4 * g + r) * a.d_v] : 0.f;

  for (int c = chunks - 1; c >= 0; --c) {
    const int tok = rg.start + c * kC, n = min(kC, rg.len - c * kC);
    const Chunk ch{seq, tok, n, c};
    const size_t unit = (size_t)(base + c) * a.heads + head;
    const T* K = static_cast<const T*>(a.k) + ((size_t)tok * a.key_heads + hk) * DK;
    const T* Q = static_cast<const T*>(a.q) + ((size_t)tok * a.key_heads + hk) * DK;
    const T* dO = static_cast<const T*>(a.dO) + ((size_t)tok * a.heads + head) * a.d_v + col;
    const float* P = reinterpret_cast<const float*>(a.ws + a.at.p) + unit * kC * (KDA ? DK : 1);
    const float* F = reinterpret_cast<const float*>(a.ws + a.at.f) + unit * kC * (KDA ? DK : 1);
    const uint16_t* Ntp =
        reinterpret_cast<const uint16_t*>(a.ws + a.at.nt_pack) + unit * (kTriFrags * 3 * kFrag);
    const uint16_t* Mtp =
        reinterpret_cast<const uint16_t*>(a.ws + a.at.m_pack) + unit * (kTriFrags * 3 * kFrag);

    float* Hc = reinterpret_cast<float*>(a.ws + a.at.grad) + unit * DK * a.d_v + col;
#pragma unroll
    for (int m = 0; m < IT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) Hc[(size_t)(16 * m + 4 * g + r) * a.d_v] = H[m][r];

    // dU = F (K H) + M^T dO
    f32x4 y[4], dq[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      y[m] = f32x4{0.f, 0.f, 0.f, 0.f};
      dq[m] = load_tile(dO, vld, m, n);
    }
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      const Frag<3> h = split_tiles<3>(H[2 * ks], H[2 * ks + 1]);
#pragma unroll
      for (int m = 0; m < 4; ++m) mma(y[m], key_rows<NT, KDA>(K, kld, F, DK, m, ks, n), h);
    }
    if (!KDA) {
#pragma unroll
      for (int m = 0; m < 4; ++m) y[m] *= row_vec(F, m);
    }
    {
      Frag<NV> x[2];
      x[0] = split_tiles<NV>(dq[0], dq[1]);
      x[1] = split_tiles<NV>(dq[2], dq[3]);
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (upper_frag(m, ks) >= 0) mma(y[m], load_pack(Mtp, upper_frag(m, ks)), x[ks]);
    }
    if (DELTA) {
      f32x4 b[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) b[m] = beta_rows(a, ch, head, m);
      Frag<3> x[2];
      x[0] = split_tiles<3>(b[0] * y[0], b[1] * y[1]);
      x[1] = split_tiles<3>(b[2] * y[2], b[3] * y[3]);
      float* Y = reinterpret_cast<float*>(a.ws + a.at.y) + unit * kC * a.d_v + col;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (upper_frag(m, ks) >= 0) mma(z, load_pack(Ntp, upper_frag(m, ks)), x[ks]);
        y[m] -= z;
        store_tile(Y, (size_t)a.d_v, m, kC, y[m]);
        y[m] *= b[m];
      }
    }
    T* dV = static_cast<T*>(a.dv) + ((size_t)tok * a.heads + head) * a.d_v + col;
#pragma unroll
    for (int m = 0; m < 4; ++m) store_tile(dV, vld, m, n, y[m]);

    // dS = P_end H + (P Q)^T dO - (P K)^T dR
    if (!KDA) {
      const float last = P[kC - 1];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const f32x4 p = row_vec(P, m);
        dq[m] *= p;
        y[m] *= -p;
      }
#pragma unroll
      for (int m = 0; m < IT; ++m) H[m] *= last;
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) y[m] = -y[m];
#pragma unroll
      for (int m = 0; m < IT; ++m) H[m] *= row_vec(P + (kC - 1) * DK, m);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Frag<3> x = split_tiles<3>(dq[2 * ks], dq[2 * ks + 1]);
      const Frag<3> z = split_tiles<3>(y[2 * ks], y[2 * ks + 1]);
#pragma unroll
      for (int m = 0; m < IT; ++m) {
        mma(H[m], key_cols<NT, KDA>(Q, kld, P, DK, m, ks, n), x);
        if (DELTA) mma(H[m], key_cols<NT, KDA>(K, kld, P, DK, m, ks, n), z);
      }
    }
  }
  if (a.dS0) {
#pragma unroll
    for (int m = 0; m < IT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) a.dS0[state + (size_t)(16 * m + 4 * g + r) * a.d_v] = H[m][r];
  }
}

template <int RULE, int DK, typename T>
hipError_t chain(const ScanArgs& a, int what, hipStream_t stream) {
  const dim3 grid((unsigned)((size_t)a.n_seq * a.heads * (a.d_v / 64))), block(256);
  if (what == 0) hipLaunchKernelGGL((forward_kernel<RULE, DK, T, false>), grid, block, 0, stream, a);
  else if (what == 1) hipLaunchKernelGGL((forward_kernel<RULE, DK, T, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((reverse_kernel<RULE, DK, T>), grid, block, 0, stream, a);
  return hipGetLastError();
}
template <int DK, typename T>
hipError_t chain_rule(const ScanArgs& a, int what, hipStream_t stream) {
  switch (a.rule) {
    case kGDN: return chain<kGDN, DK, T>(a, what, stream);
    case kKDA: return chain<kKDA, DK, T>(a, what, stream);
    default: return chain<kMAMBA2, DK, T>(a, what, stream);
  }
}
hipError_t chain_any(const ScanArgs& a, int what, hipStream_t stream) {
  if (a.d_k == 128)
    return a.bf16 ? chain_rule<128, bf16_t>(a, what, stream) : chain_rule<128, float>(a, what, stream);
  return a.bf16 ? chain_rule<64, bf16_t>(a, what, stream) : chain_rule<64, float>(a, what, stream);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_forward(const ScanArgs& a, bool save, hipStream_t stream) {
  if (a.bf16 && a.rule != kKDA) return launch_scan_chain(a, save ? 1 : 0, stream);
  return scan::chain_any(a, save ? 1 : 0, stream);
}
hipError_t launch_scan_reverse(const ScanArgs& a, hipStream_t stream) {
  if (a.bf16 && a.rule != kKDA) return launch_scan_chain(a, 2, stream);
  return scan::chain_any(a, 2, stream);
}

}  // namespace seed
