// The gradients inside each chunk, for every (chunk, head) at once, from the
// states S and H on both sides of the chunk and E and Y (formulas in
// seed_scan.h).  A gate's gradient is summed over the pairs s < t <= r that
// its decay lies between, each without the gate itself (the decays before
// and behind it), so no quotient is taken and a gate of 0 has its gradient.
#include "seed_scan_chain.h"

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

// Element (channel i, column j) of a chunk's state in the workspace.
template <int DK>
__device__ __forceinline__ int state_at(int i, int j) {
  const int m = 2 * (i >> 5) + ((i >> 2) & 1), g = (i >> 3) & 3;
  return chunk_state_at<DK>(m, g, j) + (i & 3);
}

// A chunk whose gates per key channel decay too far for quotients: the pairs
// one by one, in fp32.  Such chunks are rare; the others return at once.
template <int DK, int DV, typename T>
__global__ __launch_bounds__(256) void grads_kda_slow_kernel(ScanArgs a) {
  constexpr int NT = sizeof(T) == 2 ? 1 : 3;   // terms of an input
  extern __shared__ float lds[];
  float* dL = lds;                   // [64][65]
  float* dM = dL + kC * kLd;
  float* hs = dM + kC * kLd;         // [DK]
  const Chunk ch = chunk_of_slot(a, blockIdx.x / a.heads);
  if (ch.n == 0) return;
  const int head = head_of(a, blockIdx.x % a.heads), tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int l16 = l & 15, g16 = l >> 4, n = ch.n;
  const size_t unit = (size_t)(blockIdx.x / a.heads) * a.heads + head;
  if (!reinterpret_cast<const int*>(a.ws + a.at.slow)[unit]) return;
  const int hk = head / (a.heads / a.key_heads);
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * DV;
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* dO = static_cast<const T*>(a.dO) + ((size_t)ch.tok * a.heads + head) * DV;
  const float* P = reinterpret_cast<const float*>(a.ws + a.at.p) + unit * kC * DK;
  const float* F = reinterpret_cast<const float*>(a.ws + a.at.f) + unit * kC * DK;
  const float* Sc = reinterpret_cast<const float*>(a.ws + a.at.state) + unit * DK * DV;
  const float* Hc = reinterpret_cast<const float*>(a.ws + a.at.grad) + unit * DK * DV;
  const float* E = reinterpret_cast<const float*>(a.ws + a.at.e) + unit * kC * DV;
  const float* Y = reinterpret_cast<const float*>(a.ws + a.at.y) + unit * kC * DV;
  const float bl = l < n ? a.beta[((size_t)ch.tok + l) * a.heads + head] : 0.f;   // lane t: beta_t

  // <H, S> by key channel
  for (int i = w; i < DK; i += 4) {
    float x = 0.f;
    for (int j = l; j < DV; j += 64) x += Sc[state_at<DK>(i, j)] * Hc[state_at<DK>(i, j)];
    x = sum64(x);
    if (l == 0) hs[i] = x;
  }
  // dbeta = Y . E
  for (int t = 16 * w; t < 16 * w + 16; ++t) {
    float x = 0.f;
    for (int j = l; j < DV; j += 64) x += Y[(size_t)t * DV + j] * E[(size_t)t * DV + j];
    x = sum64(x);
    if (l == 0 && t < n) a.dbeta[((size_t)ch.tok + t) * a.heads + head] = x;
  }
  __syncthreads();

  // a fragment of rows of u or dR, and of dO (the contracted index along d_v)
  auto rows_of = [&](const float* base, int tile, int ks) {
    const int t = 16 * tile + l16;
    float x[8];
    load_row8(base + (size_t)t * DV, 32 * ks, true, x);
    const float b = __shfl(bl, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= b;
    return split<3>(x);
  };
  auto rows_do = [&](int ks) {
    const int t = 16 * w + l16;
    float x[8];
    load_row8(dO + (size_t)t * vld, 32 * ks, t < n, x);
    return split<NT>(x);
  };

  // the pairs (t, s): dL and dM
  for (int sb = 0; sb < 4; ++sb) {
    f32x4 cl = {0.f, 0.f, 0.f, 0.f}, cm = cl;
    if (sb <= w) {
#pragma unroll
      for (int ks = 0; ks < DV / 32; ++ks) {
        const Frag<3> u = rows_of(E, sb, ks);
        mma(cm, rows_do(ks), u);
        mma(cl, rows_of(Y, w, ks), u);
      }
    }
    const int s = 16 * sb + l16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * g16 + r;
      dL[t * kLd + s] = s < t ? -cl[r] : 0.f;
      dM[t * kLd + s] = s <= t ? cm[r] : 0.f;
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

  // dQ and dK: the parts through the states
  for (int it = 0; it < DK / 16; ++it) {
    const int i = 16 * it + l16;
    f32x4 x1 = {0.f, 0.f, 0.f, 0.f}, x2 = x1, x3 = x1;
    auto load_state8 = [&](const float* p, int ks, float(&x)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = p[state_at<DK>(i, 32 * ks + 16 * (j >> 2) + 4 * g16 + (j & 3))];
    };
#pragma unroll
    for (int ks = 0; ks < DV / 32; ++ks) {
      float x[8];
      load_state8(Sc, ks, x);
      const Frag<3> s = split<3>(x);
      mma(x1, rows_do(ks), s);
      mma(x2, rows_of(Y, w, ks), s);
      load_state8(Hc, ks, x);
      mma(x3, rows_of(E, w, ks), split<3>(x));
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * g16 + r;
      const float q = t < n ? load_scalar(Q + (size_t)t * kld + i) : 0.f;
      const float k = t < n ? load_scalar(K + (size_t)t * kld + i) : 0.f;
      const float p = P[t * DK + i], f = F[t * DK + i];
      tp[t * DK + i] = q * x1[r] - k * x2[r];
      tf[t * DK + i] = k * x3[r];
      if (t < n) {
        wq[(size_t)t * a.heads * DK + i] = p * x1[r];
        wk[(size_t)t * a.heads * DK + i] = f * x3[r] - p * x2[r];
      }
    }
  }

  // The pairs: a thread owns a channel and sums them one by one,
  // its group every NG-th column s.
  constexpr int NG = 256 / DK;
  float* qs = hs + DK;               // [64][DK]
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

// Rows [row][kRow] of fp32 in LDS as a left fragment contracted over columns
// 32 ks .. + 31, or the transpose.
__device__ __forceinline__ void mat_rows(const float* mat, int row, int ks, float (&x)[8]) {
  const float* at = mat + row * kRow + 32 * ks + 4 * (lane_id() >> 4);
  tiles_to_floats(*reinterpret_cast<const f32x4*>(at), *reinterpret_cast<const f32x4*>(at + 16), x);
}
__device__ __forceinline__ void mat_cols(const float* mat, int col, int ks, float (&x)[8]) {
  const float* at = mat + (32 * ks + 4 * (lane_id() >> 4)) * kRow + col;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = at[(16 * (j >> 2) + (j & 3)) * kRow];
}

// 32 channels of an array by rows of 64 bytes, pieces of 16: piece c of row t
// at c ^ (t / 4) % 4.  As a fragment: channels 16 half .. + 15, contracted over
// rows 32 ks .. + 31, by transposing reads.
__device__ __forceinline__ int part_at(int t, int c) { return t * 64 + ((c ^ ((t >> 2) & 3)) << 4); }
template <int PLANE>
__device__ __forceinline__ Frag<3> part_cols(const char* planes, int half, int ks) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const int l = lane_id(), i = l & 15, g = l >> 4;
  Frag<3> f;
#pragma unroll
  for (int m = 0; m < 3; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = 32 * ks + 16 * h + 4 * g + (i >> 2);
      const char* at = planes + m * PLANE + part_at(t, 2 * half + ((i & 3) >> 1)) + 8 * (i & 1);
      const u32x2 x = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                     (__attribute__((address_space(3))) bf16x4*)(at)));
      f.t[m][2 * h] = x[0];
      f.t[m][2 * h + 1] = x[1];
    }
  return f;
}

// Row `row` of an array in the order of load_row8, all of it on its way at
// once (a branch around each piece made every one wait for the one before);
// row n - 1 instead of a row behind it, taken for 0 by `or_zero`.
template <int KS, typename T>
__device__ __forceinline__ void load_rows(const T* base, size_t ld, int row, int n, float (&x)[KS][8]) {
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) load_row8(base + (size_t)min(row, n - 1) * ld, 32 * ks, true, x[ks]);
}
__device__ __forceinline__ void or_zero(float (&x)[8], bool live) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = live ? x[j] : 0.f;
}

// Rows t0 .. t0 + 3 (of n) of dQ and dK, channel i: to the gradients, or to
// the workspace where heads share keys.  (With scalar gates the products are
// left between these branches: behind them they spilt, 249 us instead of 232.)
template <typename T>
__device__ __forceinline__ void store_keys(const ScanArgs& a, int tok, int t0, int n, int head, int hk,
                                           int i, int d_k, const f32x4& dq, const f32x4& dk) {
  if (a.key_heads != a.heads) {
    const size_t at = ((size_t)(tok + t0) * a.heads + head) * d_k + i;
    float* q = reinterpret_cast<float*>(a.ws + a.at.dq) + at;
    float* k = reinterpret_cast<float*>(a.ws + a.at.dk) + at;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (t0 + r < n) {
        q[(size_t)r * a.heads * d_k] = dq[r];
        k[(size_t)r * a.heads * d_k] = dk[r];
      }
  } else {
    const size_t at = ((size_t)(tok + t0) * a.key_heads + hk) * d_k + i;
    T* q = static_cast<T*>(a.dq) + at;
    T* k = static_cast<T*>(a.dk) + at;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (t0 + r < n) {
        store_scalar(q + (size_t)r * a.key_heads * d_k, dq[r]);
        store_scalar(k + (size_t)r * a.key_heads * d_k, dk[r]);
      }
  }
}

// One value of N planes.
template <int DK, int N>
__device__ __forceinline__ float lds_value(const char* planes, int t, int i) {
  float x = 0.f;
#pragma unroll
  for (int n = N - 1; n >= 0; --n)
    x += __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(
             planes + n * kPlane<DK> + piece_at<DK>(t, i >> 3) + 2 * (i & 7)) << 16);
  return x;
}

// Scalar gates.  Eight waves a (chunk, head): wave (rows 16 w4, half) has the
// 16 tokens' rows of dO, dR and u in registers and every other 16 columns of
// each result.  First the pairs inside the chunk (K and Q in LDS, u of the
// other waves' rows through LDS), then 32 channels of S and H at a time.
//
// Bound by latency, one workgroup a CU (its rows alone are 112 registers a
// lane): 8192 tokens x 16 heads of 128 x 128 in bf16 take 235 us, 336 MB at
// 1.4 TB/s, matrix cores 19 % and VALU 36 % busy.  (K and Q again from memory
// behind the states' loads, to wait for both, and the rows' pieces one after
// the other: 269.)
// Four waves with all columns, so that two workgroups share a CU, spilt 100
// registers and took 357 us; four waves with the whole register file 482.
template <int RULE, int DK, int DV, typename T>
struct GradLds {
  static constexpr int NT = sizeof(T) == 2 ? 1 : 3, NE = RULE != kMAMBA2 ? 3 : NT;
  static constexpr int kq = 2 * NT * kPlane<DK>;
  static constexpr int u = 3 * (DV / 32) * NE * 1024;
  static constexpr int mats = 2 * kC * kRow * 4;
  static constexpr int plane = 32 * DV * 2;          // 32 channels of S or H, one term
  static constexpr int pairs = u > mats ? u : mats;
  static constexpr int small = kq + (pairs > 6 * plane ? pairs : 6 * plane);
  static constexpr int bytes = small + (int)sizeof(Decay) + (2 + 4 + 4) * kC * 4 + 64;
};

template <int RULE, int DK, int DV, typename T>
__global__ __launch_bounds__(512) void grads_scalar_kernel(ScanArgs a) {
  constexpr bool DELTA = RULE != kMAMBA2;
  using Lds = GradLds<RULE, DK, DV, T>;
  constexpr int NT = Lds::NT, NE = Lds::NE, KS = DV / 32, MT = DK / 32;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  char* Kp = smem;
  char* Qp = smem + NT * kPlane<DK>;
  char* Up = smem + Lds::kq;
  float* m0 = reinterpret_cast<float*>(Up);   // two fp32 matrices where u was
  float* m1 = m0 + kC * kRow;
  Decay& dec = *reinterpret_cast<Decay*>(smem + Lds::small);
  float* Pv = reinterpret_cast<float*>(smem + Lds::small + sizeof(Decay));
  float* Fv = Pv + kC;
  float* red = Fv + kC;       // [4][64]
  float* dPF = red + 4 * kC;  // [half][dP, dF][64]
  float* hs = dPF + 4 * kC;   // [8]
  const Chunk ch = chunk_of_slot(a, blockIdx.x / a.heads);
  if (ch.n == 0) return;
  const int head = head_of(a, blockIdx.x % a.heads), tid = threadIdx.x, l = lane_id(), l16 = l & 15, g = l >> 4;
  const int w4 = (tid >> 6) & 3, half = tid >> 8, n = ch.n;
  const size_t unit = (size_t)(blockIdx.x / a.heads) * a.heads + head;
  const int hk = head / (a.heads / a.key_heads);
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * DV;
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const float* Sc = reinterpret_cast<const float*>(a.ws + a.at.state) + unit * DK * DV;
  const float* Hc = reinterpret_cast<const float*>(a.ws + a.at.grad) + unit * DK * DV;

  // K and Q into LDS
  if constexpr (NT == 1) {
    async_rows<DK, 8>(K, Q, kld, n, lds_offset(Kp), lds_offset(Qp), true, wave_id());
  } else {
    for (int i = tid; i < 2 * kC * (DK / 8); i += 512) {
      const int which = i / (kC * (DK / 8)), t = i / (DK / 8) % kC, c = i % (DK / 8);
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (t < n) {
        const T* from = (which ? Q : K) + (size_t)t * kld + 8 * c;
        float y[4], z[4];
        load_vec<4>(from, y);
        load_vec<4>(from + 4, z);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = y[r];
          x[4 + r] = z[r];
        }
      }
      const Frag<NT> f = split<NT>(x);
#pragma unroll
      for (int m = 0; m < NT; ++m)
        *reinterpret_cast<u32x4*>((which ? Qp : Kp) + m * kPlane<DK> + piece_at<DK>(t, c)) = f.t[m];
    }
  }
  // the wave's rows of dO, dR and u
  const int row = 16 * w4 + l16;
  Frag<NT> ado[KS];
  Frag<3> adr[DELTA ? KS : 1];
  Frag<NE> au[KS];
  {
    const bool live = row < n;
    const size_t vat = ((size_t)ch.tok * a.heads + head) * DV, vld = (size_t)a.heads * DV, eat = unit * kC * DV;
    const float b = DELTA ? reinterpret_cast<const float*>(a.ws + a.at.vec)[unit * 256 + 128 + row] : 0.f;
    float db = 0.f;
    float o[KS][8], x[KS][8], y[DELTA ? KS : 1][8];
    load_rows(static_cast<const T*>(a.dO) + vat, vld, row, n, o);
    if constexpr (DELTA) {
      load_rows(reinterpret_cast<const float*>(a.ws + a.at.e) + eat, DV, row, n, x);
      load_rows(reinterpret_cast<const float*>(a.ws + a.at.y) + eat, DV, row, n, y);
    } else {
      load_rows(static_cast<const T*>(a.v) + vat, vld, row, n, x);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      or_zero(o[ks], live);
      or_zero(x[ks], live);
      ado[ks] = split<NT>(o[ks]);
      if constexpr (DELTA) {
        or_zero(y[ks], live);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          db += x[ks][j] * y[ks][j];
          x[ks][j] *= b;
          y[ks][j] *= b;
        }
        adr[ks] = split<3>(y[ks]);
      }
      au[ks] = split<NE>(x[ks]);
      if (w4 < 3 && half == 0) {
#pragma unroll
        for (int m = 0; m < NE; ++m)
          *reinterpret_cast<u32x4*>(Up + (((w4 * KS + ks) * NE + m) * 64 + l) * 16) = au[ks].t[m];
      }
    }
    if (DELTA) {   // dbeta = Y . E
      db += __shfl_xor(db, 16);
      db += __shfl_xor(db, 32);
      if (half == 0 && g == 0 && live) a.dbeta[((size_t)ch.tok + row) * a.heads + head] = db;
    }
  }
  if (tid < 64) {
    const float gate = tid < n ? a.g[((size_t)ch.tok + tid) * a.heads + head] : 1.f;
    float P, F;
    decays(dec, gate, P, F);
    Pv[tid] = P;
    Fv[tid] = F;
  }
  if (tid < 4 * kC) red[tid] = 0.f;
  async_wait();
  __syncthreads();

  // the pairs: row tile w4, column tiles b = half, half + 2
  f32x4 pl[2], pm[2], pw[2], pg[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int b = 2 * i + half;
    pl[i] = pm[i] = pw[i] = pg[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (b > w4) continue;
    f32x4 kk = pl[i], qk = pl[i];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Frag<NE> u = au[ks];
      if (b < w4) {
#pragma unroll
        for (int m = 0; m < NE; ++m)
          u.t[m] = *reinterpret_cast<const u32x4*>(Up + (((b * KS + ks) * NE + m) * 64 + l) * 16);
      }
      mma(pm[i], ado[ks], u);
      if constexpr (DELTA) mma(pl[i], adr[ks], u);
    }
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      const Frag<NT> k = lds_rows<DK, NT>(Kp, b, ks);
      if (DELTA) mma(kk, lds_rows<DK, NT>(Kp, w4, ks), k);
      mma(qk, lds_rows<DK, NT>(Qp, w4, ks), k);
    }
    const int t = 16 * w4 + 4 * g, s = 16 * b + l16;
    if (b < w4) {
      pg[i] = *reinterpret_cast<const f32x4*>(dec.pre + t) * (dec.suf[s] * dec.mid[4 * w4 + b]);
    } else {
      pg[i] = inside<true>(dec.gate, t, s);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (s > t + r) pg[i][r] = pm[i][r] = 0.f;
        if (s >= t + r) pl[i][r] = 0.f;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) pw[i][r] = s < t + r ? pm[i][r] * qk[r] - pl[i][r] * kk[r] : 0.f;
    pl[i] *= -pg[i];
    pm[i] *= pg[i];
  }
  __syncthreads();
  auto put = [&](float* mat, int i, const f32x4& x) {
    const int b = 2 * i + half;
#pragma unroll
    for (int r = 0; r < 4; ++r) mat[(16 * w4 + 4 * g + r) * kRow + 16 * b + l16] = x[r];
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    put(m0, i, pg[i]);
    put(m1, i, pw[i]);
  }
  __syncthreads();
  // dg from the pairs: sum over r >= t > s of G_rt W_rs G_{t-1,s}
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int b = 2 * i + half, t = 16 * b + l16;
    if (b > w4) continue;
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    for (int ks = 0; ks <= (b >> 1); ++ks) {
      float x[8], y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      mat_rows(m1, 16 * w4 + l16, ks, x);
      if (t > 0) mat_rows(m0, t - 1, ks, y);
      mma(d, split<3>(x), split<3>(y));
    }
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) sum += d[r] * pg[i][r];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (g == 0) red[w4 * kC + t] = sum;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    put(m0, i, pl[i]);
    put(m1, i, pm[i]);
  }
  __syncthreads();

  // dQ and dK from the pairs; column tiles it = half, half + 2, ...
  f32x4 dq[MT], dk[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) dq[i] = dk[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    float x[8], y[8];
    Frag<3> fm, ft, fl;
    const bool low = ks <= (w4 >> 1), up = ks >= (w4 >> 1);
    if (low) {
      mat_rows(m1, row, ks, x);
      fm = split<3>(x);
    }
    if (up) {
      mat_cols(m1, row, ks, x);
      ft = split<3>(x);
    }
    if (DELTA) {
      mat_rows(m0, row, ks, x);
      mat_cols(m0, row, ks, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] += y[j];
      fl = split<3>(x);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int it = 2 * i + half;
      const Frag<NT> k = lds_channels<DK, NT>(Kp, it, ks);
      if (low) mma(dq[i], fm, k);
      if (up) mma(dk[i], ft, lds_channels<DK, NT>(Qp, it, ks));
      if (DELTA) mma(dk[i], fl, k);
    }
  }

  // through the states, 32 channels at a time: rows of 8 values a thread
  const bool stager = tid < 4 * DV;
  float sv[8], hv[8], hsum = 0.f;
  auto fetch = [&](int part) {
    if (!stager) return;
    float y[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = chunk_state_at<DK>(2 * part + h, tid & 3, tid >> 2);
      load_vec<4>(Sc + at, y);
#pragma unroll
      for (int r = 0; r < 4; ++r) sv[4 * h + r] = y[r];
      load_vec<4>(Hc + at, y);
#pragma unroll
      for (int r = 0; r < 4; ++r) hv[4 * h + r] = y[r];
    }
  };
  fetch(0);
  f32x4 dp = {0.f, 0.f, 0.f, 0.f}, df = dp;
  const f32x4 pt = *reinterpret_cast<const f32x4*>(Pv + 16 * w4 + 4 * g);
  const f32x4 ft = *reinterpret_cast<const f32x4*>(Fv + 16 * w4 + 4 * g);
  const bool shared = a.key_heads != a.heads;
#pragma unroll
  for (int part = 0; part < MT; ++part) {
    __syncthreads();
    if (stager) {
      const int at = part_at(tid >> 2, tid & 3);
      const Frag<3> s = split<3>(sv), h = split<3>(hv);
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        *reinterpret_cast<u32x4*>(Up + m * Lds::plane + at) = s.t[m];
        *reinterpret_cast<u32x4*>(Up + (3 + m) * Lds::plane + at) = h.t[m];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) hsum += sv[j] * hv[j];
    }
    __syncthreads();
    if (part + 1 < MT) fetch(part + 1);
    // channels 32 part + 16 half + l16
    f32x4 x1 = {0.f, 0.f, 0.f, 0.f}, x2 = x1, x3 = x1;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag<3> s = part_cols<Lds::plane>(Up, half, ks);
      const Frag<3> h = part_cols<Lds::plane>(Up + 3 * Lds::plane, half, ks);
      mma(x1, ado[ks], s);
      if constexpr (DELTA) mma(x2, adr[ks], s);
      mma(x3, au[ks], h);
    }
    const int i = 32 * part + 16 * half + l16;
    dq[part] += pt * x1;
    dk[part] += ft * x3 - pt * x2;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w4 + 4 * g + r;
      if (t >= n) continue;
      // (from LDS: a load would wait for the next part's states, loads arriving in order)
      const float q = lds_value<DK, NT>(Qp, t, i), k = lds_value<DK, NT>(Kp, t, i);
      dp[r] += q * x1[r] - k * x2[r];
      df[r] += k * x3[r];
      if (shared) {
        const size_t at = ((size_t)(ch.tok + t) * a.heads + head) * DK + i;
        reinterpret_cast<float*>(a.ws + a.at.dq)[at] = dq[part][r];
        reinterpret_cast<float*>(a.ws + a.at.dk)[at] = dk[part][r];
      } else {
        const size_t at = ((size_t)(ch.tok + t) * a.key_heads + hk) * DK + i;
        store_scalar(static_cast<T*>(a.dq) + at, dq[part][r]);
        store_scalar(static_cast<T*>(a.dk) + at, dk[part][r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float x = sum16(dp[r]), y = sum16(df[r]);
    if (l16 == 0) {
      dPF[half * 2 * kC + 16 * w4 + 4 * g + r] = x;
      dPF[half * 2 * kC + kC + 16 * w4 + 4 * g + r] = y;
    }
  }
  hsum = sum64(hsum);
  if (l == 0) hs[tid >> 6] = hsum;
  __syncthreads();
  if (tid >= 64) return;
  // and from the states: c_t = dP_t + g_{t+1} c_{t+1} behind t (<H, S> at the
  // end), b_{t+1} = g_t b_t + dF_t before it
  const float gate = dec.gate[tid];
  float A = __shfl_down(gate, 1), B = dPF[tid] + dPF[2 * kC + tid];
  if (tid == 63) A = 1.f;
  float A2 = gate, B2 = dPF[kC + tid] + dPF[3 * kC + tid];
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const float ax = __shfl_down(A, o), bx = __shfl_down(B, o);
    const float ay = __shfl_up(A2, o), by = __shfl_up(B2, o);
    if (tid + o < 64) {
      B += A * bx;
      A *= ax;
    }
    if (tid >= o) {
      B2 += A2 * by;
      A2 *= ay;
    }
  }
  const float all = ((hs[0] + hs[1]) + (hs[2] + hs[3])) + ((hs[4] + hs[5]) + (hs[6] + hs[7]));
  const float c = B + A * all, b0 = __shfl_up(B2, 1), b = tid ? b0 : 0.f;
  const float before = tid ? Pv[tid - 1] : 1.f;
  const float pairs = (red[tid] + red[kC + tid]) + (red[2 * kC + tid] + red[3 * kC + tid]);
  if (tid < n)
    a.dg[((size_t)ch.tok + tid) * a.heads + head] = pairs + (c * before + Fv[tid] * b);
}

// Gates per key channel, chunks whose P lies in kSafe .. 1 / kSafe and whose
// gates are 1/4 and more (the others are marked and left to the kernel above).
// With K~ = P K, Q~ = P Q, K' = K / P:
//   dQ = P (dO S^T + dM K'),  dK = P (dL K' - dR S^T) + F (u H^T)
//        + (dL^T K~ + dM^T Q~) / P
// and with the parts of k.dK in this order called row, end and col,
//   g_t dg_t = sum over r >= t of (q.dQ + row - col)_r + sum over s < t of
//   end_s + P_end <H, S>, channel by channel: the pairs that lie behind t
// cancel in the first sum, which is why small gates take the other way.
//
// Four waves, one a SIMD, with the whole register file: a wave's 16 rows of
// dO, dR and u and its rows and columns of dL and dM are fragments for all
// channels (eight waves with half of the columns each spilt 97 registers and
// split the triangles anew for every 32 channels: 312 us for 3001 tokens x 16
// heads of 128 x 128 instead of 203; loads without branches, all on their way
// at once, and one loop body, not four, made that 170).  Bound by latency:
// matrix cores 11 %, VALU 24 % busy.
template <int DK, int DV, typename T>
struct KdaLds {
  static constexpr int NT = sizeof(T) == 2 ? 1 : 3;
  static constexpr int u = 3 * (DV / 32) * 3 * 1024;
  static constexpr int mats = 2 * kC * kRow * 4;
  static constexpr int plane = 32 * DV * 2, kplane = kC * 64;   // 32 channels of S or H, of K
  static constexpr int s = u > mats ? u : mats;
  static constexpr int k = s + 6 * plane;
  static constexpr int small = k + 9 * kplane;
  static constexpr int bytes = small + (4 * 2 * 32 + 4 * 32 + 8) * 4;
};

template <int DK, int DV, typename T>
__global__ __launch_bounds__(256, 1) void grads_kda_kernel(ScanArgs a) {
  using Lds = KdaLds<DK, DV, T>;
  constexpr int NT = Lds::NT, KS = DV / 32, MT = DK / 32;
  constexpr int NS = DV / 64;                   // columns of a state a thread brings
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  float* m0 = reinterpret_cast<float*>(smem);   // u of the waves, then dL and dM
  float* m1 = m0 + kC * kRow;
  char* Sp = smem + Lds::s;
  char* Kp = smem + Lds::k;                     // K', K~, Q~: three planes each
  float* tot = reinterpret_cast<float*>(smem + Lds::small);   // [x, z][4][32]
  float* hs = tot + 4 * 2 * 32;                 // [wave][32]
  int* bad = reinterpret_cast<int*>(hs + 4 * 32);
  const Chunk ch = chunk_of_slot(a, blockIdx.x / a.heads);
  if (ch.n == 0) return;
  const int head = head_of(a, blockIdx.x % a.heads), tid = threadIdx.x, l = lane_id(), l16 = l & 15, g = l >> 4;
  const int w = wave_id(), n = ch.n;
  const size_t unit = (size_t)(blockIdx.x / a.heads) * a.heads + head;
  const int hk = head / (a.heads / a.key_heads);
  const size_t kld = (size_t)a.key_heads * DK, gld = (size_t)a.heads * DK;
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const float* gates = a.g + ((size_t)ch.tok * a.heads + head) * DK;
  const float* P = reinterpret_cast<const float*>(a.ws + a.at.p) + unit * kC * DK;
  const float* F = reinterpret_cast<const float*>(a.ws + a.at.f) + unit * kC * DK;
  const float* Sc = reinterpret_cast<const float*>(a.ws + a.at.state) + unit * DK * DV;
  const float* Hc = reinterpret_cast<const float*>(a.ws + a.at.grad) + unit * DK * DV;

  if (tid == 0) *bad = 0;
  __syncthreads();
  {
    bool fine = true;
    constexpr int CHECKS = kC * DK / 4 / 256;
    f32x4 p[CHECKS], gt[CHECKS];
    float k[CHECKS][4];
#pragma unroll
    for (int c = 0; c < CHECKS; ++c) {   // (rows behind the last: the last again)
      const int e = tid + 256 * c, t = e / (DK / 4), i = 4 * (e % (DK / 4)), live = min(t, n - 1);
      p[c] = *reinterpret_cast<const f32x4*>(P + t * DK + i);
      gt[c] = *reinterpret_cast<const f32x4*>(gates + (size_t)live * gld + i);
      load_vec<4>(K + (size_t)live * kld + i, k[c]);
    }
#pragma unroll
    for (int c = 0; c < CHECKS; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        fine &= p[c][r] >= kSafe && p[c][r] <= 1.f / kSafe && gt[c][r] >= 0.25f && fabsf(k[c][r]) <= 0x1p40f;
    if (!fine) *bad = 1;
  }
  // the wave's rows of dO, dR and u
  const int row = 16 * w + l16;
  Frag<NT> ado[KS];
  Frag<3> adr[KS], au[KS];
  float db = 0.f;
  {
    const bool live = row < n;
    const size_t eat = unit * kC * DV;
    const float b = reinterpret_cast<const float*>(a.ws + a.at.vec)[unit * 256 + 128 + row];
    float o[KS][8], x[KS][8], y[KS][8];
    load_rows(static_cast<const T*>(a.dO) + ((size_t)ch.tok * a.heads + head) * DV, (size_t)a.heads * DV, row, n, o);
    load_rows(reinterpret_cast<const float*>(a.ws + a.at.e) + eat, DV, row, n, x);
    load_rows(reinterpret_cast<const float*>(a.ws + a.at.y) + eat, DV, row, n, y);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      or_zero(o[ks], live);
      or_zero(x[ks], live);
      or_zero(y[ks], live);
      ado[ks] = split<NT>(o[ks]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        db += x[ks][j] * y[ks][j];
        x[ks][j] *= b;
        y[ks][j] *= b;
      }
      adr[ks] = split<3>(y[ks]);
      au[ks] = split<3>(x[ks]);
      if (w < 3) {
#pragma unroll
        for (int m = 0; m < 3; ++m)
          *reinterpret_cast<u32x4*>(smem + (((w * KS + ks) * 3 + m) * 64 + l) * 16) = au[ks].t[m];
      }
    }
    db += __shfl_xor(db, 16);
    db += __shfl_xor(db, 32);
  }
  __syncthreads();
  if (tid == 0) reinterpret_cast<int*>(a.ws + a.at.slow)[unit] = *bad;
  if (*bad) return;
  if (g == 0 && row < n) a.dbeta[((size_t)ch.tok + row) * a.heads + head] = db;

  // the pairs: row tile w
  f32x4 pl[4], pm[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    pl[b] = pm[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (b > w) continue;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Frag<3> u = au[ks];
      if (b < w) {
#pragma unroll
        for (int m = 0; m < 3; ++m)
          u.t[m] = *reinterpret_cast<const u32x4*>(smem + (((b * KS + ks) * 3 + m) * 64 + l) * 16);
      }
      mma(pm[b], ado[ks], u);
      mma(pl[b], adr[ks], u);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 4 * g + r;
      if (b == w && l16 > t) pm[b][r] = 0.f;
      pl[b][r] = b == w && l16 >= t ? 0.f : -pl[b][r];
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m0[(16 * w + 4 * g + r) * kRow + 16 * b + l16] = pl[b][r];
      m1[(16 * w + 4 * g + r) * kRow + 16 * b + l16] = pm[b][r];
    }
  __syncthreads();
  // their rows and columns w as fragments
  Frag<3> rl[2], rm[2], cl[2], cm[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    float x[8];
    if (ks <= (w >> 1)) {
      mat_rows(m0, row, ks, x);
      rl[ks] = split<3>(x);
      mat_rows(m1, row, ks, x);
      rm[ks] = split<3>(x);
    }
    if (ks >= (w >> 1)) {
      mat_cols(m0, row, ks, x);
      cl[ks] = split<3>(x);
      mat_cols(m1, row, ks, x);
      cm[ks] = split<3>(x);
    }
  }

  float sv[NS][8], hv[NS][8], pv[8];
  Piece<T> kv, qv;
  auto fetch = [&](int part) {
    float y[4];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = chunk_state_at<DK>(2 * part + h, tid & 3, 64 * i + (tid >> 2));
        load_vec<4>(Sc + at, y);
#pragma unroll
        for (int r = 0; r < 4; ++r) sv[i][4 * h + r] = y[r];
        load_vec<4>(Hc + at, y);
#pragma unroll
        for (int r = 0; r < 4; ++r) hv[i][4 * h + r] = y[r];
      }
    const int t = tid >> 2, c = 32 * part + 8 * (tid & 3);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load_vec<4>(P + t * DK + c + 4 * h, y);
#pragma unroll
      for (int r = 0; r < 4; ++r) pv[4 * h + r] = y[r];
    }
    kv.clear();
    qv.clear();
    if (t < n) {
      kv.load(K + (size_t)t * kld + c);
      qv.load(Q + (size_t)t * kld + c);
    }
  };
  fetch(0);
#pragma unroll 1
  for (int part = 0; part < MT; ++part) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int at = part_at(64 * i + (tid >> 2), tid & 3);
      const Frag<3> s = split<3>(sv[i]), h = split<3>(hv[i]);
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        *reinterpret_cast<u32x4*>(Sp + m * Lds::plane + at) = s.t[m];
        *reinterpret_cast<u32x4*>(Sp + (3 + m) * Lds::plane + at) = h.t[m];
      }
    }
    // <H, S> by channel: a wave's 16 NS columns
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x = sv[0][j] * hv[0][j];
      if (NS == 2) x += sv[NS - 1][j] * hv[NS - 1][j];
#pragma unroll
      for (int o = 4; o < 64; o *= 2) x += __shfl_xor(x, o);
      if (l < 4) hs[w * 32 + 8 * l + j] = x;
    }
    {
      float x[8], y[8], z[8];
      kv.get(y);
      qv.get(z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = y[j] * __builtin_amdgcn_rcpf(pv[j]);
        y[j] *= pv[j];
        z[j] *= pv[j];
      }
      const int at = part_at(tid >> 2, tid & 3);
      const Frag<3> f0 = split<3>(x), f1 = split<3>(y), f2 = split<3>(z);
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        *reinterpret_cast<u32x4*>(Kp + m * Lds::kplane + at) = f0.t[m];
        *reinterpret_cast<u32x4*>(Kp + (3 + m) * Lds::kplane + at) = f1.t[m];
        *reinterpret_cast<u32x4*>(Kp + (6 + m) * Lds::kplane + at) = f2.t[m];
      }
    }
    __syncthreads();
    if (part + 1 < MT) fetch(part + 1);
    const int t0 = 16 * w + 4 * g;
    float q[2][4], k[2][4], pt[2][4], ft[2][4], gt[2][4], end[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = 32 * part + 16 * half + l16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = t0 + r;
        pt[half][r] = P[t * DK + i];
        ft[half][r] = F[t * DK + i];
        const size_t live = min(t, n - 1);
        q[half][r] = load_scalar(Q + live * kld + i);
        k[half][r] = load_scalar(K + live * kld + i);
        gt[half][r] = gates[live * gld + i];
      }
      end[half] = P[(kC - 1) * DK + i];
    }
    f32x4 x1[2], x2[2], x3[2], a1[2], a2[2], a3[2];
#pragma unroll
    for (int half = 0; half < 2; ++half)
      x1[half] = x2[half] = x3[half] = a1[half] = a2[half] = a3[half] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const Frag<3> s = part_cols<Lds::plane>(Sp, half, ks);
        const Frag<3> h = part_cols<Lds::plane>(Sp + 3 * Lds::plane, half, ks);
        mma(x1[half], ado[ks], s);
        mma(x2[half], adr[ks], s);
        mma(x3[half], au[ks], h);
      }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (ks <= (w >> 1)) {
          const Frag<3> f = part_cols<Lds::kplane>(Kp, half, ks);
          mma(a1[half], rm[ks], f);
          mma(a2[half], rl[ks], f);
        }
        if (ks >= (w >> 1)) {
          mma(a3[half], cl[ks], part_cols<Lds::kplane>(Kp + 3 * Lds::kplane, half, ks));
          mma(a3[half], cm[ks], part_cols<Lds::kplane>(Kp + 6 * Lds::kplane, half, ks));
        }
      }
    float xs[2][4], zs[2][4], bx[2], bz[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = 32 * part + 16 * half + l16;
      end[half] *= (hs[16 * half + l16] + hs[32 + 16 * half + l16]) +
                   (hs[64 + 16 * half + l16] + hs[96 + 16 * half + l16]);
      f32x4 dq, dk;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float p = pt[half][r], rk = p * (a2[half][r] - x2[half][r]);
        const float ck = a3[half][r] * __builtin_amdgcn_rcpf(p), fk = ft[half][r] * x3[half][r];
        dq[r] = p * (x1[half][r] + a1[half][r]);
        dk[r] = rk + ck + fk;
        xs[half][r] = t0 + r < n ? q[half][r] * dq[r] + k[half][r] * (rk - ck) : 0.f;
        zs[half][r] = t0 + r < n ? k[half][r] * fk : 0.f;
      }
      store_keys<T>(a, ch.tok, t0, n, head, hk, i, DK, dq, dk);
      // sums of x over t and behind, of z before t: rows, lanes, waves
      const float sx = (xs[half][0] + xs[half][1]) + (xs[half][2] + xs[half][3]);
      const float sz = (zs[half][0] + zs[half][1]) + (zs[half][2] + zs[half][3]);
      float allx = sx, allz = sz;
      bx[half] = bz[half] = 0.f;
#pragma unroll
      for (int o = 1; o < 4; ++o) {
        const float x = __shfl(sx, (l16 + 16 * (g + o)) & 63), z = __shfl(sz, (l16 + 16 * (g - o)) & 63);
        bx[half] += g + o < 4 ? x : 0.f;
        bz[half] += g - o >= 0 ? z : 0.f;
      }
      allx += __shfl_xor(allx, 16);
      allx += __shfl_xor(allx, 32);
      allz += __shfl_xor(allz, 16);
      allz += __shfl_xor(allz, 32);
      if (g == 0) {
        tot[w * 32 + 16 * half + l16] = allx;
        tot[128 + w * 32 + 16 * half + l16] = allz;
      }
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = 32 * part + 16 * half + l16;
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        bx[half] += o > w ? tot[o * 32 + 16 * half + l16] : 0.f;
        bz[half] += o < w ? tot[128 + o * 32 + 16 * half + l16] : 0.f;
      }
#pragma unroll
      for (int r = 3; r >= 0; --r) {
        bx[half] += xs[half][r];
        xs[half][r] = bx[half];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = t0 + r;
        if (t < n)
          a.dg[((size_t)(ch.tok + t) * a.heads + head) * DK + i] =
              (xs[half][r] + bz[half] + end[half]) * __builtin_amdgcn_rcpf(gt[half][r]);
        bz[half] += zs[half][r];
      }
    }
  }
}

// Gradients of keys and queries that several heads share: the sum over the
// group in head order.  Rows outside every sequence are left as they were.
// Bound by HBM (42 MB in 13.5 us).
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
  const dim3 grid((unsigned)((size_t)a.slots * a.heads));
  hipError_t e;
  if constexpr (RULE != kKDA) {
    constexpr size_t bytes = GradLds<RULE, DK, DV, T>::bytes;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(grads_scalar_kernel<RULE, DK, DV, T>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((grads_scalar_kernel<RULE, DK, DV, T>), grid, dim3(512), bytes, stream, a);
  } else {
    constexpr size_t bytes = KdaLds<DK, DV, T>::bytes;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(grads_kda_kernel<DK, DV, T>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return e;
    constexpr size_t slow = (2 * kC * kLd + DK + 3 * kC * DK) * sizeof(float);
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(grads_kda_slow_kernel<DK, DV, T>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)slow);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((grads_kda_kernel<DK, DV, T>), grid, dim3(256), bytes, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((grads_kda_slow_kernel<DK, DV, T>), grid, dim3(256), slow, stream, a);
  }
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
