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

// A chunk's rows of a float32 array into three planes, rows from n on 0: a
// thread's pieces, all on their way at once.
template <int DK>
struct FloatRows {
  static constexpr int N = kC * DK / 8 / 256;
  f32x4 a[N], b[N];
  __device__ __forceinline__ void load(const float* rows, size_t ld, int n) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x + 256 * i, t = e / (DK / 8), c = e % (DK / 8);
      const float* p = rows + (size_t)min(t, n - 1) * ld + 8 * c;
      a[i] = *reinterpret_cast<const f32x4*>(p);
      b[i] = *reinterpret_cast<const f32x4*>(p + 4);
    }
  }
  __device__ __forceinline__ void split_to(int n, char* planes) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x + 256 * i, t = e / (DK / 8), c = e % (DK / 8);
      float x[8];
      tiles_to_floats(a[i], b[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = t < n ? x[j] : 0.f;
      const Frag<3> f = split<3>(x);
#pragma unroll
      for (int m = 0; m < 3; ++m)
        *reinterpret_cast<u32x4*>(planes + m * kPlane<DK> + piece_at<DK>(t, c)) = f.t[m];
    }
  }
};

// Four waves a (chunk, head); wave w has the tokens 16 w .. + 15 as rows.  K
// and Q lie in LDS by whole rows (256 bytes at a time: fragments straight from
// memory, 64 bytes of a row at a time, took the preparation of 64 x 512
// tokens x 16 heads 132 us), L then in their place.  (float32: only K, in
// three terms; a wave takes its rows of Q from memory.)
//
// Bound by the steps' latency and the VALU, not by memory: for those 64 x 512
// tokens x 16 heads 127 us, 461 MB moved at 3.6 TB/s, the VALU issuing half of
// the time and the matrix cores 13 % of it; the decays are one wave's work and
// the inverses of L's diagonal blocks 16 dependent steps.  Four workgroups a
// CU hide part of it.
template <int RULE, int DK, typename T, bool BWD>
__global__ __launch_bounds__(256) void prep_scalar_kernel(ScanArgs a) {
  constexpr int NT = sizeof(T) == 2 ? 1 : 3;
  constexpr bool DELTA = RULE != kMAMBA2;
  constexpr int KQ = (NT == 1 ? 2 : 3) * kPlane<DK>, SOLVE = (kC * kRow + 64 * 20) * 4;
  __shared__ __attribute__((aligned(1024))) char buf[DELTA && SOLVE > KQ ? SOLVE : KQ];
  __shared__ __attribute__((aligned(16))) float bt[kC];
  __shared__ Decay dec;
  char* Kp = buf;
  char* Qp = buf + kPlane<DK>;
  float* L = reinterpret_cast<float*>(buf);
  const Chunk ch = chunk_of_slot(a, blockIdx.x / a.heads);
  if (ch.n == 0) return;
  const int head = head_of(a, blockIdx.x % a.heads), w = wave_id(), l = lane_id(), g16 = l >> 4, l16 = l & 15;
  const size_t unit = (size_t)(blockIdx.x / a.heads) * a.heads + head;
  const int hk = head / (a.heads / a.key_heads);
  const size_t ld = (size_t)a.key_heads * DK;
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  uint16_t* mp = reinterpret_cast<uint16_t*>(a.ws + a.at.m_pack) + unit * (kTriFrags * 3 * kFrag);

  // loads arrive in order, and the decays are the longest way: the gates first
  const int row = 16 * w + l16;
  float gate = 1.f, beta = 0.f;
  if (w == 0) {
    const size_t at = ((size_t)ch.tok + min(l, ch.n - 1)) * a.heads + head;
    gate = a.g[at];
    if (DELTA) beta = a.beta[at];
  }
  float q[NT == 1 ? 1 : DK / 32][8];   // the wave's rows of Q (float32)
  if constexpr (NT == 1) {
    async_rows<DK, 4>(K, Q, ld, ch.n, lds_offset(Kp), lds_offset(Qp), true, w);
  } else {
    FloatRows<DK> k;
    k.load(K, ld, ch.n);
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) load_piece(Q + (size_t)min(row, ch.n - 1) * ld, 32 * ks, true, q[ks]);
    k.split_to(ch.n, Kp);
  }
  if (w == 0) {
    float P, F;
    float* vec = reinterpret_cast<float*>(a.ws + a.at.vec) + unit * 256;
    if (DELTA) {
      bt[l] = l < ch.n ? beta : 0.f;
      vec[128 + l] = bt[l];
    }
    decays(dec, l < ch.n ? gate : 1.f, P, F);
    vec[l] = P;
    vec[64 + l] = F;
  }
  async_wait();
  __syncthreads();

  // lane (t, s): its row of the right operand and four rows of the left;
  // backward the left operand is Q, and M's tile comes out transposed
  f32x4 lt[4], mt[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) lt[b] = mt[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < DK / 32; ++ks) {
    const Frag<NT> kt = lds_rows<DK, NT>(Kp, w, ks);
    Frag<NT> qt;
    if constexpr (NT == 1) {
      qt = lds_rows<DK, NT>(Qp, w, ks);
    } else {
      for (int j = 0; j < 8; ++j) q[ks][j] = row < ch.n ? q[ks][j] : 0.f;
      qt = split<NT>(q[ks]);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b > w) continue;
      const Frag<NT> kb = lds_rows<DK, NT>(Kp, b, ks);
      if (DELTA) mma(lt[b], kb, kt);
      if (BWD) mma(mt[b], qt, kb);
      else mma(mt[b], kb, qt);
    }
  }
  if (DELTA) __syncthreads();   // L takes K's place
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    f32x4 gl = {0.f, 0.f, 0.f, 0.f}, gm = gl, mm = mt[b];
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
        const bool in = BWD ? sm <= tm + r : s + r <= t;
        gm[r] = in ? gm[r] : 0.f;
        mm[r] = in ? mm[r] : 0.f;
        gl[r] = s + r < t ? gl[r] : 0.f;
      }
    }
    // (rows and columns past the sequence's end repeat its last token: their
    // beta, values and read-outs are dropped, but N and M must not reach them)
    if (ch.n < kC) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (t >= ch.n || s + r >= ch.n) gl[r] = lt[b][r] = 0.f;
        if (BWD ? tm + r >= ch.n || sm >= ch.n : t >= ch.n || s + r >= ch.n) gm[r] = mm[r] = 0.f;
      }
    }
    if (DELTA) *reinterpret_cast<f32x4*>(L + t * kRow + s) = lt[b] * gl;
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
    solve(L, L + kC * kRow, bt, w);
    uint16_t* np = reinterpret_cast<uint16_t*>(a.ws + a.at.n_pack) + unit * (kTriFrags * 3 * kFrag);
    for (int i = w; i < 8; i += 4) pack_triangle(np, L, false, i >> 1, i & 1);
    if (BWD) {
      uint16_t* tp =
          reinterpret_cast<uint16_t*>(a.ws + a.at.nt_pack) + unit * (kTriFrags * 3 * kFrag);
      for (int i = w; i < 8; i += 4) pack_triangle(tp, L, true, i >> 1, i & 1);
    }
  }
}

// Gates per key channel.  With P the decay from the chunk's start,
// G_ts = P_t / P_s channel by channel, so L and M are products of K P, Q P and
// K / P.  That is taken where every P of the chunk lies in 2^-60 .. 2^60 (the
// hardware reciprocal is good to a unit in the last place, 2^-23, and a masked
// pair stays finite).  bf16 rows of K and Q come whole through LDS (182 us for
// 24 ragged sequences of 7919 tokens in all, 32 heads of 128 x 128; loads of
// the lanes' own 64-byte pieces and an IEEE division cost 30 more).  Chunks with
// smaller decays, zeros among them, are summed pair by pair (slow_triangles).

// The product over the lanes of a row of 16 up to (and with) this one.
__device__ __forceinline__ float row_prefix(float x) {
#define SEED_STEP(CTRL)                                                                       \
  x *= __int_as_float(__builtin_amdgcn_update_dpp(0x3f800000, __float_as_int(x), CTRL, 0xf, 0xf, \
                                                  false))
  SEED_STEP(0x111);   // row_shr 1, 2, 4, 8
  SEED_STEP(0x112);
  SEED_STEP(0x114);
  SEED_STEP(0x118);
#undef SEED_STEP
  return x;
}

// L and M [64][kRow] (M only for s <= t) and P, F of a chunk, any gates: lane
// s runs down column s, a wave has 16 rows; 16 channels at a time through
// `buf` (3 * 64 * 17 floats).
template <int DK, typename T>
__device__ void slow_triangles(const T* __restrict__ K, const T* __restrict__ Q, size_t ld,
                               const float* __restrict__ gates, size_t gld, int n, float* buf,
                               float* L, float* M, float* __restrict__ P, float* __restrict__ F) {
  constexpr int LR = 17;
  float* gs = buf;
  float* kk = gs + kC * LR;
  float* qq = kk + kC * LR;
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  float accL[16], accM[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) accL[t] = accM[t] = 0.f;
  for (int c0 = 0; c0 < DK; c0 += 16) {
    __syncthreads();
    for (int e = tid; e < kC * 16; e += 256) {
      const int t = e >> 4, i = e & 15;
      const bool live = t < n;
      gs[t * LR + i] = live ? gates[(size_t)t * gld + c0 + i] : 1.f;
      kk[t * LR + i] = live ? load_scalar(K + (size_t)t * ld + c0 + i) : 0.f;
      qq[t * LR + i] = live ? load_scalar(Q + (size_t)t * ld + c0 + i) : 0.f;
    }
    __syncthreads();
    if (tid < 16) {
      float x = 1.f;
#pragma unroll 1
      for (int t = 0; t < kC; ++t) {
        x *= gs[t * LR + tid];
        P[t * DK + c0 + tid] = x;
      }
      x = 1.f;
#pragma unroll 1
      for (int t = kC - 1; t >= 0; --t) {
        F[t * DK + c0 + tid] = x;
        x *= gs[t * LR + tid];
      }
    }
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const float ks = kk[l * LR + i];
      float cur = 0.f;
#pragma unroll 1
      for (int t = 0; t < 16 * w; ++t) cur = t > l ? cur * gs[t * LR + i] : (t == l ? ks : 0.f);
#pragma unroll
      for (int o = 0; o < 16; ++o) {
        const int t = 16 * w + o;
        cur = t > l ? cur * gs[t * LR + i] : (t == l ? ks : 0.f);
        accL[o] += kk[t * LR + i] * cur;
        accM[o] += qq[t * LR + i] * cur;
      }
    }
  }
#pragma unroll
  for (int o = 0; o < 16; ++o) {
    const int t = 16 * w + o;
    L[t * kRow + l] = l < t ? accL[o] : 0.f;
    M[t * kRow + l] = accM[o];
  }
  __syncthreads();
}

// Four waves a (chunk, head); wave w has the tokens 16 w .. + 15 as rows.
template <int DK, typename T, bool BWD>
__global__ __launch_bounds__(256, 2) void prep_kda_kernel(ScanArgs a) {
  constexpr int KS = DK / 32;
  // K and Q as they come (bf16), then K / P in fragments, then L and the
  // inverses (or, pair by pair, L, M and 16 channels)
  constexpr int KBAR = 4 * KS * 3 * kFrag * 2, MAT = kC * kRow * 4, SLOW = 2 * MAT + 3 * kC * 17 * 4;
  __shared__ __attribute__((aligned(1024))) char buf[KBAR > SLOW ? KBAR : SLOW];
  __shared__ __attribute__((aligned(16))) float tot[4][DK];
  __shared__ __attribute__((aligned(16))) float bt[kC];
  __shared__ int unsafe;
  uint16_t* kl = reinterpret_cast<uint16_t*>(buf);
  float* L = reinterpret_cast<float*>(buf);
  float* M = L + kC * kRow;
  float* X = M + kC * kRow;
  const Chunk ch = chunk_of_slot(a, blockIdx.x / a.heads);
  if (ch.n == 0) return;
  const int head = head_of(a, blockIdx.x % a.heads), tid = threadIdx.x, w = wave_id(), l = lane_id();
  const int g16 = l >> 4, l16 = l & 15;
  const size_t unit = (size_t)(blockIdx.x / a.heads) * a.heads + head;
  const int hk = head / (a.heads / a.key_heads);
  const size_t ld = (size_t)a.key_heads * DK, gld = (size_t)a.heads * DK;
  const T* K = static_cast<const T*>(a.k) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)ch.tok * a.key_heads + hk) * DK;
  const float* gates = a.g + ((size_t)ch.tok * a.heads + head) * DK;
  float* P = reinterpret_cast<float*>(a.ws + a.at.p) + unit * kC * DK;
  float* F = reinterpret_cast<float*>(a.ws + a.at.f) + unit * kC * DK;
  uint16_t* mp = reinterpret_cast<uint16_t*>(a.ws + a.at.m_pack) + unit * (kTriFrags * 3 * kFrag);

  if constexpr (sizeof(T) == 2)
    async_rows<DK, 4>(K, Q, ld, ch.n, lds_offset(buf), lds_offset(buf + kPlane<DK>), true, w);
  const int t0 = 16 * w + l16;
  const bool live = t0 < ch.n;
  float p[KS][8], k[KS][8], q[KS][8];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    load_piece(gates + (size_t)t0 * gld, 32 * ks, live, p[ks]);
    if constexpr (sizeof(T) == 4) {
      load_piece(K + (size_t)t0 * ld, 32 * ks, live, k[ks]);
      load_piece(Q + (size_t)t0 * ld, 32 * ks, live, q[ks]);
    }
  }
  if (tid < kC) {
    bt[tid] = tid < ch.n ? a.beta[((size_t)ch.tok + tid) * a.heads + head] : 0.f;
    reinterpret_cast<float*>(a.ws + a.at.vec)[unit * 256 + 128 + tid] = bt[tid];
  }
  if (tid == 0) unsafe = 0;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[ks][j] = row_prefix(live ? p[ks][j] : 1.f);
    if (l16 == 15) {
      float* to = &tot[w][32 * ks + 8 * g16];
      *reinterpret_cast<f32x4*>(to) = f32x4{p[ks][0], p[ks][1], p[ks][2], p[ks][3]};
      *reinterpret_cast<f32x4*>(to + 4) = f32x4{p[ks][4], p[ks][5], p[ks][6], p[ks][7]};
    }
  }
  async_wait();
  __syncthreads();
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag<1> x = lds_rows<DK, 1>(buf, w, ks), y = lds_rows<DK, 1>(buf + kPlane<DK>, w, ks);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k[ks][2 * j] = live ? __uint_as_float(x.t[0][j] << 16) : 0.f;
        k[ks][2 * j + 1] = live ? __uint_as_float(x.t[0][j] & 0xffff0000u) : 0.f;
        q[ks][2 * j] = live ? __uint_as_float(y.t[0][j] << 16) : 0.f;
        q[ks][2 * j + 1] = live ? __uint_as_float(y.t[0][j] & 0xffff0000u) : 0.f;
      }
    }
    __syncthreads();   // K / P takes their place
  }
  bool fine = true;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    f32x4 before[2], all[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      before[h] = all[h] = f32x4{1.f, 1.f, 1.f, 1.f};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(&tot[b][32 * ks + 8 * g16 + 4 * h]);
        if (b < w) before[h] *= x;
        all[h] *= x;
      }
    }
    float end[8], kb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = p[ks][j] * before[j >> 2][j & 3], inv = __builtin_amdgcn_rcpf(x);
      fine &= x >= kSafe && inv >= kSafe;
      p[ks][j] = x;
      end[j] = all[j >> 2][j & 3] * inv;
      kb[j] = k[ks][j] * inv;
      fine &= fabsf(kb[j]) <= 0x1p100f;   // no overflow in a masked pair
      k[ks][j] *= x;
      q[ks][j] *= x;
    }
    const Frag<3> f = split<3>(kb);
#pragma unroll
    for (int m = 0; m < 3; ++m)
      *reinterpret_cast<u32x4*>(kl + (((w * KS + ks) * 3 + m) * 64 + l) * 8) = f.t[m];
    float* to = P + t0 * DK + 32 * ks + 8 * g16;
    *reinterpret_cast<f32x4*>(to) = f32x4{p[ks][0], p[ks][1], p[ks][2], p[ks][3]};
    *reinterpret_cast<f32x4*>(to + 4) = f32x4{p[ks][4], p[ks][5], p[ks][6], p[ks][7]};
    to = F + t0 * DK + 32 * ks + 8 * g16;
    *reinterpret_cast<f32x4*>(to) = f32x4{end[0], end[1], end[2], end[3]};
    *reinterpret_cast<f32x4*>(to + 4) = f32x4{end[4], end[5], end[6], end[7]};
  }
  if (!fine) unsafe = 1;
  __syncthreads();

  if (unsafe) {
    slow_triangles<DK>(K, Q, ld, gates, gld, ch.n, X, L, M, P, F);
    for (int i = w; i < 8; i += 4) pack_triangle(mp, M, BWD, i >> 1, i & 1);
  } else {
    f32x4 lt[4], mt[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) lt[b] = mt[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag<3> kt = split<3>(k[ks]), qt = split<3>(q[ks]);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b > w) continue;
        Frag<3> kb;
#pragma unroll
        for (int m = 0; m < 3; ++m)
          kb.t[m] = *reinterpret_cast<const u32x4*>(kl + (((b * KS + ks) * 3 + m) * 64 + l) * 8);
        mma(lt[b], kb, kt);
        if (BWD) mma(mt[b], qt, kb);
        else mma(mt[b], kb, qt);
      }
    }
    __syncthreads();   // L takes the place of K / P
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      f32x4 ll = lt[b], mm = mt[b];
      if (b == w) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          ll[r] = 4 * g16 + r < l16 ? ll[r] : 0.f;
          mm[r] = (BWD ? l16 <= 4 * g16 + r : 4 * g16 + r <= l16) ? mm[r] : 0.f;
        }
      }
      *reinterpret_cast<f32x4*>(L + (16 * w + l16) * kRow + 16 * b + 4 * g16) = ll;
      if (BWD) {
        if (upper_frag(b, w >> 1) >= 0) store_half(mp, upper_frag(b, w >> 1), w & 1, mm);
      } else {
        if (lower_frag(w, b >> 1) >= 0) store_half(mp, lower_frag(w, b >> 1), b & 1, mm);
      }
    }
    __syncthreads();
  }
  solve(L, X, bt, w);
  uint16_t* np = reinterpret_cast<uint16_t*>(a.ws + a.at.n_pack) + unit * (kTriFrags * 3 * kFrag);
  for (int i = w; i < 8; i += 4) pack_triangle(np, L, false, i >> 1, i & 1);
  if (BWD) {
    uint16_t* tp =
        reinterpret_cast<uint16_t*>(a.ws + a.at.nt_pack) + unit * (kTriFrags * 3 * kFrag);
    for (int i = w; i < 8; i += 4) pack_triangle(tp, L, true, i >> 1, i & 1);
  }
}

template <int DK, typename T, bool BWD>
hipError_t prep(const ScanArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((size_t)a.slots * a.heads));
  if (a.rule == kKDA) {
    hipLaunchKernelGGL((prep_kda_kernel<DK, T, BWD>), grid, dim3(256), 0, stream, a);
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
