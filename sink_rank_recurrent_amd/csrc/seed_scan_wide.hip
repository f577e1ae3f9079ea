// The recurrence from chunk to chunk, and back, where a key operand needs
// more than one bf16 term: float32 inputs, and gates per key channel (K and
// Q are scaled by the decays channel by channel).  As in seed_scan_chain.hip a
// wave owns 16 columns; the operands are split into LDS planes by the whole
// workgroup, from values loaded while the chunk before was computed.  With
// gates per channel K serves twice, scaled by P and by F: the second fills
// the same planes once the first is used up, and F is loaded once P is used
// (held together with P it spilt, and every spilt value was waited for: 25000
// cycles a chunk of 48000).  P_end waits in LDS for the same reason: held in
// registers from before the corrections on, 24 sequences of 7919 tokens took
// 514 us with their preparation, 413 so.  A barrier behind the last use of N, M and the
// vectors lets the next chunk's be loaded while the state is brought up.
//
// Bound as there: 24 ragged sequences of 7919 tokens x 32 heads with gates per
// channel take 306 us forward (matrix cores 40 %, VALU 37 % busy, 1.5 TB/s:
// the longest sequences' workgroups run on alone); 5 sequences of 3001 tokens
// x 16 heads 137 us forward and 205 us backward in 160 workgroups, the
// chain's latency.  float32, 16384 tokens x 16 heads of 64 x 64 in segments of
// 16 chunks: 99 us for the segments' carries and 105 us for the read-outs.
#include "seed_scan_chain.h"

namespace seed {
namespace scan {
namespace {

// A thread's share of a 64 x DK operand: PPT pieces.
template <int DK, int THREADS>
constexpr int kShare = kC * DK / 8 / THREADS;
template <int DK, int THREADS, typename T>
struct Share {
  Piece<T> x[kShare<DK, THREADS>];
  // rows from n on are 0
  __device__ __forceinline__ void load(const T* base, size_t ld, int n) {
#pragma unroll
    for (int i = 0; i < kShare<DK, THREADS>; ++i) {
      const int e = i * THREADS + threadIdx.x, t = e / (DK / 8), c = e % (DK / 8);
      if (t < n) x[i].load(base + (size_t)t * ld + 8 * c);
      else x[i].clear();
    }
  }
};
// x (times `scale`) into N planes.
template <int DK, int THREADS, int N, bool SCALED, typename T>
__device__ __forceinline__ void fill(char* planes, const Share<DK, THREADS, T>& v,
                                     const Share<DK, THREADS, float>& scale) {
#pragma unroll
  for (int i = 0; i < kShare<DK, THREADS>; ++i) {
    const int e = i * THREADS + threadIdx.x, t = e / (DK / 8), c = e % (DK / 8);
    float x[8];
    v.x[i].get(x);
    if (SCALED) {
      float y[8];
      scale.x[i].get(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= y[j];
    }
    const Frag<N> f = split<N>(x);
#pragma unroll
    for (int n = 0; n < N; ++n)
      *reinterpret_cast<u32x4*>(planes + n * kPlane<DK> + piece_at<DK>(t, c)) = f.t[n];
  }
}

template <typename T>
struct Tiles {
  T x[4][4];
  __device__ __forceinline__ void load(const T* p, size_t ld, uint32_t lane, int n) {
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const T* row = p + (size_t)(16 * m + r) * ld;
        x[m][r] = n >= kC || 16 * m + 4 * (lane_id() >> 4) + r < n ? row[lane] : T(0);
      }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) x[m][r] = T(0);
  }
  __device__ __forceinline__ f32x4 tile(int m) const {
    return f32x4{load_scalar(&x[m][0]), load_scalar(&x[m][1]), load_scalar(&x[m][2]),
                 load_scalar(&x[m][3])};
  }
};

template <int RULE, int DK, typename T, bool READ>
struct Wide {
  static constexpr bool KDA = RULE == kKDA, DELTA = RULE != kMAMBA2;
  static constexpr int NV = sizeof(T) == 2 ? 1 : 3;              // a value or a gradient
  static constexpr int q = 3 * kPlane<DK>;
  static constexpr int n = q + (READ ? 3 * kPlane<DK> : 0);
  static constexpr int m = n + (DELTA ? kTriFrags * 3 * 1024 : 0);
  static constexpr int vec = m + (READ ? kTriFrags * 3 * 1024 : 0);
  static constexpr int end = vec + 1024;   // KDA: the last 256 values of P, P_end behind them
  static constexpr int bytes = end + (KDA ? 1024 : 0);
};

template <int RULE, int DK, int NW, typename T, int MODE>
__global__ __launch_bounds__(64 * NW) void wide_forward_kernel(ScanArgs a) {
  constexpr bool READ = MODE == kRead, SAVE = MODE == kSave, CARRY = MODE == kCarry;
  using W = Wide<RULE, DK, T, READ>;
  constexpr bool KDA = W::KDA, DELTA = W::DELTA;
  constexpr int IT = DK / 16, TH = 64 * NW;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int w = wave_id();
  const Walk<NW> at(a, a.d_v + (CARRY && DELTA ? DK : 0));
  if (at.c0 > at.c1 || (CARRY && at.c1 == at.chunks)) return;   // nothing is behind a last segment
  const uint32_t lds0 = lds_offset(lds);
  const Range rg = at.rg;
  const int c0 = at.c0, c1 = at.c1, base = at.base;
  const bool unit_cols = CARRY && DELTA && at.col0 >= a.d_v;
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * a.d_v;
  const size_t state = ((size_t)at.seq * a.heads + at.head) * DK * a.d_v;
  const uint32_t g = lane_id() >> 4, row_lane = 4 * g * (uint32_t)vld + at.col;
  const uint32_t keep_lane = 4 * g * a.d_v + at.col, state_lane = 8 * g * a.d_v + at.col;
  const T* K = static_cast<const T*>(a.k) + ((size_t)rg.start * a.key_heads + at.hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)rg.start * a.key_heads + at.hk) * DK;
  const size_t vat = ((size_t)rg.start * a.heads + at.head) * a.d_v;
  const T* V = static_cast<const T*>(a.v) + vat;
  T* out = static_cast<T*>(a.o) + vat;

  f32x4 S[IT];
  if (unit_cols) unit_state(at.col - a.d_v, S);
  else if (!CARRY && at.split)
    load_chunk_state(reinterpret_cast<const float*>(a.ws + a.at.start) + at.segment * DK * a.d_v, at.col0, S);
  else load_state(!CARRY && a.S0 ? a.S0 + state : nullptr, a.d_v, state_lane, S);
  float through = 1.f;

  Share<DK, TH, T> kr, qr;
  Share<DK, TH, float> xr;   // P, then F
  constexpr bool OWN = sizeof(T) == 2 || NW == 4;   // room for the waves' own columns of V
  char* mine = lds + W::bytes + kOwn<T> * w;
  const uint32_t mine0 = lds0 + W::bytes + kOwn<T> * w;
  Tiles<T> v;
  auto keys = [&](int c) {
    const int n = min(kC, rg.len - c * kC);
    kr.load(K + (size_t)c * kC * kld, kld, n);
    if (READ) qr.load(Q + (size_t)c * kC * kld, kld, n);
    if (KDA)
      xr.load(reinterpret_cast<const float*>(a.ws + a.at.p) +
                  ((size_t)(base + c) * a.heads + at.head) * kC * DK, DK, kC);
  };
  auto values = [&](int c) {
    const int n = min(kC, rg.len - c * kC);
    if (unit_cols) return;
    if constexpr (OWN) wave_load(V + at.col0 + (size_t)c * kC * vld, vld, n, mine0);
    else v.load(V + (size_t)c * kC * vld, vld, row_lane, n);
  };
  auto triangles = [&](int c) {
    const size_t unit = (size_t)(base + c) * a.heads + at.head;
    constexpr size_t pack = kTriFrags * 3 * kFrag;
    if (DELTA)
      async_pack<NW>(reinterpret_cast<const uint16_t*>(a.ws + a.at.n_pack) + unit * pack, lds0 + W::n, w);
    if (READ)
      async_pack<NW>(reinterpret_cast<const uint16_t*>(a.ws + a.at.m_pack) + unit * pack, lds0 + W::m, w);
    if (w == NW - 1) async_copy(a.ws + a.at.vec + unit * 1024, lane_id() * 16, lds0 + W::vec);
    if (KDA && w == 0)
      async_copy(a.ws + a.at.p + (unit + 1) * (kC * DK * 4) - 1024, lane_id() * 16, lds0 + W::end);
  };
  if (c0 < c1) {
    keys(c0);
    values(c0);
    triangles(c0);
  }
  for (int c = c0; c < c1; ++c) {
    const int n = min(kC, rg.len - c * kC);
    const size_t unit = (size_t)(base + c) * a.heads + at.head;
    __syncthreads();   // the chunk before is done with the planes
    if (KDA) {
      if (DELTA) fill<DK, TH, 3, true>(lds, kr, xr);
      if (READ) fill<DK, TH, 3, true>(lds + W::q, qr, xr);
    } else {
      fill<DK, TH, 3, false>(lds, kr, xr);
      if (READ) fill<DK, TH, 3, false>(lds + W::q, qr, xr);
    }
    async_wait();
    __syncthreads();
    if (SAVE)
      keep_chunk_state(reinterpret_cast<float*>(a.ws + a.at.state) + unit * DK * a.d_v, at.col0, S);
    if (KDA) xr.load(reinterpret_cast<const float*>(a.ws + a.at.f) + unit * kC * DK, DK, kC);
    else if (c + 1 < c1) keys(c + 1);

    f32x4 R[4], O[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) R[m] = O[m] = zero4();
    if (DELTA || READ) {
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        const Frag<3> s = split_tiles<3>(S[2 * ks], S[2 * ks + 1]);
        if (DELTA) {
          Frag<3> f[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) f[m] = lds_rows<DK, 3>(lds, m, ks);
          mma_tiles(R, f, s);
        }
        if (READ) {
          Frag<3> f[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) f[m] = lds_rows<DK, 3>(lds + W::q, m, ks);
          mma_tiles(O, f, s);
        }
      }
    }
    if (KDA) {   // K's planes are used up: F K takes their place
      __syncthreads();
      fill<DK, TH, 3, true>(lds, kr, xr);
      if (c + 1 < c1) keys(c + 1);
    }
    f32x4 u[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if constexpr (OWN) u[m] = unit_cols ? zero4() : wave_tile<T>(mine, m);
      else u[m] = unit_cols ? zero4() : v.tile(m);
    }
    drop_rows(u, n);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 p = KDA ? f32x4{1.f, 1.f, 1.f, 1.f} : lds_vec(lds + W::vec, m);
      if (DELTA) u[m] -= p * R[m];
      O[m] *= p;
    }
    if (DELTA) {
      f32x4 b[4], y[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        b[m] = lds_vec(lds + W::vec + 512, m);
        y[m] = zero4();
      }
      const Frag<3> x0 = split_tiles<3>(b[0] * u[0], b[1] * u[1]);
      const Frag<3> x1 = split_tiles<3>(b[2] * u[2], b[3] * u[3]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_pack<3>(lds + W::n, lower_frag(m, 0));
      mma_tiles(y, f, x0);
      f32x4 z[2] = {y[2], y[3]};
      const Frag<3> h[2] = {lds_pack<3>(lds + W::n, lower_frag(2, 1)),
                             lds_pack<3>(lds + W::n, lower_frag(3, 1))};
      mma_tiles(z, h, x1);
      u[0] -= y[0];
      u[1] -= y[1];
      u[2] -= z[0];
      u[3] -= z[1];
      drop_rows(u, n);
      if (SAVE)
        keep_tiles(reinterpret_cast<float*>(a.ws + a.at.e) + unit * kC * a.d_v, a.d_v, keep_lane, u);
#pragma unroll
      for (int m = 0; m < 4; ++m) u[m] *= b[m];
    }
    if (READ) {
      constexpr int NU = DELTA ? 3 : W::NV;   // V itself is one term
      const Frag<NU> x0 = split_tiles<NU>(u[0], u[1]), x1 = split_tiles<NU>(u[2], u[3]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_pack<3>(lds + W::m, lower_frag(m, 0));
      mma_tiles(O, f, x0);
      f32x4 z[2] = {O[2], O[3]};
      const Frag<3> h[2] = {lds_pack<3>(lds + W::m, lower_frag(2, 1)),
                             lds_pack<3>(lds + W::m, lower_frag(3, 1))};
      mma_tiles(z, h, x1);
      O[2] = z[0];
      O[3] = z[1];
      if constexpr (OWN) wave_store(out + at.col0 + (size_t)c * kC * vld, vld, n, O, mine);
      else store_tiles(out + (size_t)c * kC * vld, vld, row_lane, n, O);
    }
    if (c + 1 < c1) values(c + 1);
    // S' = P_end S + (F K)^T u
    if (KDA) {
#pragma unroll
      for (int m = 0; m < IT; ++m)
        S[m] *= *reinterpret_cast<const f32x4*>(lds + W::end + 4 * (256 - DK + state_row(m)));
    } else {
      const float end = *reinterpret_cast<const float*>(lds + W::vec + 4 * (kC - 1));
#pragma unroll
      for (int m = 0; m < 4; ++m) u[m] *= lds_vec(lds + W::vec + 256, m);
#pragma unroll
      for (int m = 0; m < IT; ++m) S[m] *= end;
      if (CARRY && !DELTA) through *= end;
    }
    __syncthreads();   // F K is in place, N, M and the vectors are used up
    if (c + 1 < c1) triangles(c + 1);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Frag<3> x = split_tiles<3>(u[2 * ks], u[2 * ks + 1]);
#pragma unroll
      for (int mm = 0; mm < IT; mm += 4) {
        Frag<3> f[4];
        f32x4 s[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          f[m] = lds_cols<DK, 3>(lds, mm + m, ks);
          s[m] = S[mm + m];
        }
        mma_tiles(s, f, x);
#pragma unroll
        for (int m = 0; m < 4; ++m) S[mm + m] = s[m];
      }
    }
  }
  if (READ && c1 == at.chunks) keep_state(a.S + state, a.d_v, state_lane, S);
  if (CARRY) {
    float* trans = reinterpret_cast<float*>(a.ws + a.at.trans);
    if (unit_cols) keep_chunk_state(trans + at.segment * DK * DK, at.col0 - a.d_v, S);
    else keep_chunk_state(reinterpret_cast<float*>(a.ws + a.at.carry) + at.segment * DK * a.d_v, at.col0, S);
    if (!DELTA && threadIdx.x == 0) trans[at.segment] = through;
  }
}

template <int DK, int RULE>
struct WideBack {
  static constexpr bool DELTA = RULE != kMAMBA2;
  static constexpr int q = 3 * kPlane<DK>;
  static constexpr int n = 2 * q;
  static constexpr int m = n + (DELTA ? kTriFrags * 3 * 1024 : 0);
  static constexpr int vec = m + kTriFrags * 3 * 1024;
  static constexpr int bytes = vec + 1024;
};

// The chunks from the last to the first (see chain_reverse_kernel).
template <int RULE, int DK, int NW, typename T, bool LOCAL>
__global__ __launch_bounds__(64 * NW) void wide_reverse_kernel(ScanArgs a) {
  using W = WideBack<DK, RULE>;
  constexpr bool KDA = RULE == kKDA, DELTA = RULE != kMAMBA2;
  constexpr int IT = DK / 16, TH = 64 * NW, NV = sizeof(T) == 2 ? 1 : 3;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int w = wave_id();
  const Walk<NW> at(a, a.d_v);
  if (at.c0 > at.c1 || (LOCAL && at.c0 == 0)) return;   // nothing is before a first segment
  const uint32_t lds0 = lds_offset(lds);
  const Range rg = at.rg;
  const int c0 = at.c0, c1 = at.c1, base = at.base;
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * a.d_v;
  const size_t state = ((size_t)at.seq * a.heads + at.head) * DK * a.d_v;
  const uint32_t g = lane_id() >> 4, row_lane = 4 * g * (uint32_t)vld + at.col;
  const uint32_t keep_lane = 4 * g * a.d_v + at.col, state_lane = 8 * g * a.d_v + at.col;
  const T* K = static_cast<const T*>(a.k) + ((size_t)rg.start * a.key_heads + at.hk) * DK;
  const T* Q = static_cast<const T*>(a.q) + ((size_t)rg.start * a.key_heads + at.hk) * DK;
  const size_t vat = ((size_t)rg.start * a.heads + at.head) * a.d_v;
  const T* dO = static_cast<const T*>(a.dO) + vat;
  T* dV = static_cast<T*>(a.dv) + vat;

  f32x4 H[IT];
  // in the segments' own first pass the last one starts from dS
  if (at.split && !LOCAL)
    load_chunk_state(reinterpret_cast<const float*>(a.ws + a.at.start) + at.segment * DK * a.d_v, at.col0, H);
  else load_state(c1 == at.chunks && a.dS ? a.dS + state : nullptr, a.d_v, state_lane, H);

  Share<DK, TH, T> kr, qr;
  Share<DK, TH, float> pr, fr;
  constexpr bool OWN = sizeof(T) == 2 || NW == 4;   // room for the waves' own columns of dO
  char* mine = lds + W::bytes + kOwn<T> * w;
  const uint32_t mine0 = lds0 + W::bytes + kOwn<T> * w;
  Tiles<T> d;
  auto keys = [&](int c) {
    const int n = min(kC, rg.len - c * kC);
    const size_t unit = (size_t)(base + c) * a.heads + at.head;
    kr.load(K + (size_t)c * kC * kld, kld, n);
    qr.load(Q + (size_t)c * kC * kld, kld, n);
    if (KDA) {
      pr.load(reinterpret_cast<const float*>(a.ws + a.at.p) + unit * kC * DK, DK, kC);
      fr.load(reinterpret_cast<const float*>(a.ws + a.at.f) + unit * kC * DK, DK, kC);
    }
  };
  auto values = [&](int c) {
    const int n = min(kC, rg.len - c * kC);
    if constexpr (OWN) wave_load(dO + at.col0 + (size_t)c * kC * vld, vld, n, mine0);
    else d.load(dO + (size_t)c * kC * vld, vld, row_lane, n);
  };
  auto triangles = [&](int c) {
    const size_t unit = (size_t)(base + c) * a.heads + at.head;
    constexpr size_t pack = kTriFrags * 3 * kFrag;
    if (DELTA)
      async_pack<NW>(reinterpret_cast<const uint16_t*>(a.ws + a.at.nt_pack) + unit * pack, lds0 + W::n, w);
    async_pack<NW>(reinterpret_cast<const uint16_t*>(a.ws + a.at.m_pack) + unit * pack, lds0 + W::m, w);
    if (w == NW - 1) async_copy(a.ws + a.at.vec + unit * 1024, lane_id() * 16, lds0 + W::vec);
  };
  if (c0 < c1) {
    keys(c1 - 1);
    values(c1 - 1);
    triangles(c1 - 1);
  }
  for (int c = c1 - 1; c >= c0; --c) {
    const int n = min(kC, rg.len - c * kC);
    const size_t unit = (size_t)(base + c) * a.heads + at.head;
    __syncthreads();
    if (KDA) {
      fill<DK, TH, 3, true>(lds, kr, fr);
      fill<DK, TH, 3, true>(lds + W::q, qr, pr);
    } else {
      fill<DK, TH, 3, false>(lds, kr, pr);
      fill<DK, TH, 3, false>(lds + W::q, qr, pr);
    }
    async_wait();
    __syncthreads();
    f32x4 y[4], go[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      y[m] = zero4();
      if constexpr (OWN) go[m] = wave_tile<T>(mine, m);
      else go[m] = d.tile(m);
    }
    drop_rows(go, n);
    if (!LOCAL)
      keep_chunk_state(reinterpret_cast<float*>(a.ws + a.at.grad) + unit * DK * a.d_v, at.col0, H);
    // P again for P K: not held through the product, which would spill it
    if (KDA) pr.load(reinterpret_cast<const float*>(a.ws + a.at.p) + unit * kC * DK, DK, kC);
    else if (c > c0) keys(c - 1);

    // dU = F (K H) + M^T dO
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      const Frag<3> h = split_tiles<3>(H[2 * ks], H[2 * ks + 1]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_rows<DK, 3>(lds, m, ks);
      mma_tiles(y, f, h);
    }
    f32x4 last[KDA ? IT : 1];
    if (KDA) {   // F K is used up: P K takes its place
#pragma unroll
      for (int m = 0; m < IT; ++m)
        last[m] = *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(a.ws + a.at.p) +
                                                  (unit * kC + kC - 1) * DK + state_row(m));
      __syncthreads();
      fill<DK, TH, 3, true>(lds, kr, pr);
      if (c > c0) keys(c - 1);
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) y[m] *= lds_vec(lds + W::vec + 256, m);
    }
    {
      const Frag<NV> x0 = split_tiles<NV>(go[0], go[1]), x1 = split_tiles<NV>(go[2], go[3]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_pack<3>(lds + W::m, upper_frag(m, 1));
      mma_tiles(y, f, x1);
      f32x4 z[2] = {y[0], y[1]};
      const Frag<3> h[2] = {lds_pack<3>(lds + W::m, upper_frag(0, 0)),
                            lds_pack<3>(lds + W::m, upper_frag(1, 0))};
      mma_tiles(z, h, x0);
      y[0] = z[0];
      y[1] = z[1];
    }
    if (DELTA) {
      f32x4 b[4], t[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        b[m] = lds_vec(lds + W::vec + 512, m);
        t[m] = zero4();
      }
      const Frag<3> x0 = split_tiles<3>(b[0] * y[0], b[1] * y[1]);
      const Frag<3> x1 = split_tiles<3>(b[2] * y[2], b[3] * y[3]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_pack<3>(lds + W::n, upper_frag(m, 1));
      mma_tiles(t, f, x1);
      f32x4 z[2] = {t[0], t[1]};
      const Frag<3> h[2] = {lds_pack<3>(lds + W::n, upper_frag(0, 0)),
                            lds_pack<3>(lds + W::n, upper_frag(1, 0))};
      mma_tiles(z, h, x0);
      y[0] -= z[0];
      y[1] -= z[1];
      y[2] -= t[2];
      y[3] -= t[3];
      drop_rows(y, n);
      if (!LOCAL)
        keep_tiles(reinterpret_cast<float*>(a.ws + a.at.y) + unit * kC * a.d_v, a.d_v, keep_lane, y);
#pragma unroll
      for (int m = 0; m < 4; ++m) y[m] *= b[m];
    }
    if (!LOCAL) {
      if constexpr (OWN) wave_store(dV + at.col0 + (size_t)c * kC * vld, vld, n, y, mine);
      else store_tiles(dV + (size_t)c * kC * vld, vld, row_lane, n, y);
    }
    if (c > c0) values(c - 1);

    // dS = P_end H + (P Q)^T dO - (P K)^T dR
    if (KDA) {
#pragma unroll
      for (int m = 0; m < 4; ++m) y[m] = -y[m];
#pragma unroll
      for (int m = 0; m < IT; ++m) H[m] *= last[m];
    } else {
      const float end = *reinterpret_cast<const float*>(lds + W::vec + 4 * (kC - 1));
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const f32x4 p = lds_vec(lds + W::vec, m);
        go[m] *= p;
        y[m] *= -p;
      }
#pragma unroll
      for (int m = 0; m < IT; ++m) H[m] *= end;
    }
    __syncthreads();   // P K is in place, N, M and the vectors are used up
    if (c > c0) triangles(c - 1);
    constexpr int NG = KDA ? NV : 3;   // dO itself, or times P
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Frag<NG> x = split_tiles<NG>(go[2 * ks], go[2 * ks + 1]);
      const Frag<3> z = split_tiles<3>(y[2 * ks], y[2 * ks + 1]);
#pragma unroll
      for (int mm = 0; mm < IT; mm += 4) {
        Frag<3> f[4];
        f32x4 s[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          f[m] = lds_cols<DK, 3>(lds + W::q, mm + m, ks);
          s[m] = H[mm + m];
        }
        mma_tiles(s, f, x);
        if (DELTA) {
#pragma unroll
          for (int m = 0; m < 4; ++m) f[m] = lds_cols<DK, 3>(lds, mm + m, ks);
          mma_tiles(s, f, z);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) H[mm + m] = s[m];
      }
    }
  }
  if (LOCAL)
    keep_chunk_state(reinterpret_cast<float*>(a.ws + a.at.carry) + at.segment * DK * a.d_v, at.col0, H);
  else if (c0 == 0 && a.dS0) keep_state(a.dS0 + state, a.d_v, state_lane, H);
}

template <typename F>
hipError_t launch(F kernel, const ScanArgs& a, int columns, int waves, size_t lds, hipStream_t stream) {
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)walk_grid(a, columns, waves)), dim3(64 * waves), lds, stream, a);
  return hipGetLastError();
}

template <int RULE, int DK, int NW, typename T>
hipError_t wide(const ScanArgs& a, int what, hipStream_t stream) {
  constexpr size_t own = sizeof(T) == 2 || NW == 4 ? kOwn<T> * NW : 0;
  constexpr size_t read = Wide<RULE, DK, T, true>::bytes + own, save = Wide<RULE, DK, T, false>::bytes + own;
  constexpr size_t back = WideBack<DK, RULE>::bytes + own;
  static_assert(read <= 160 * 1024 && save <= 160 * 1024 && back <= 160 * 1024, "LDS of a CU");
  // (segments are walked by four waves: walk_waves)
  if constexpr (NW == 4) {
    if (what == 3)
      return launch(wide_forward_kernel<RULE, DK, NW, T, kCarry>, a, a.d_v + (RULE != kMAMBA2 ? DK : 0), NW, save, stream);
    if (what == 4) return launch(wide_reverse_kernel<RULE, DK, NW, T, true>, a, a.d_v, NW, back, stream);
  }
  switch (what) {
    case 0: return launch(wide_forward_kernel<RULE, DK, NW, T, kRead>, a, a.d_v, NW, read, stream);
    case 1: return launch(wide_forward_kernel<RULE, DK, NW, T, kSave>, a, a.d_v, NW, save, stream);
    case 2: return launch(wide_reverse_kernel<RULE, DK, NW, T, false>, a, a.d_v, NW, back, stream);
    default: return hipErrorInvalidValue;
  }
}
template <int RULE, typename T>
hipError_t wide_shape(const ScanArgs& a, int what, hipStream_t stream) {
  if (a.d_k == 64) return wide<RULE, 64, 4, T>(a, what, stream);
  return walk_waves(a) == 4 ? wide<RULE, 128, 4, T>(a, what, stream)
                            : wide<RULE, 128, 8, T>(a, what, stream);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_wide(const ScanArgs& a, int what, hipStream_t stream) {
  using namespace scan;
  if (a.rule == kKDA)
    return a.bf16 ? wide_shape<kKDA, bf16_t>(a, what, stream) : wide_shape<kKDA, float>(a, what, stream);
  return a.rule == kGDN ? wide_shape<kGDN, float>(a, what, stream)
                        : wide_shape<kMAMBA2, float>(a, what, stream);
}

}  // namespace seed
