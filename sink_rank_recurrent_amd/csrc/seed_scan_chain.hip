// The recurrence from chunk to chunk, and back, for bf16 inputs and scalar
// gates (Gated DeltaNet, Mamba-2).  Columns of the state do not mix: a wave
// owns 16 of them and carries them through a sequence's chunks in its
// accumulators; every product's result is the next one's right operand in
// the registers it is already in (seed_scan.h).  The left operands (K, Q, N,
// M) are the same for all waves: they come through LDS, the next chunk's by
// asynchronous loads while this one is computed.
//
// Bound by instruction issue where the chip is full: 64 sequences x 512 tokens
// x 16 heads of 128 x 128 forward in 289 us, the matrix cores busy 46 % and
// the VALU 46 % of the time, 558 MB at 1.9 TB/s.  With fewer than 256
// workgroups (4 sequences x 2048 tokens: 128) by the chain itself, 4 us a
// chunk forward and 6.5 backward (128 and 209 us for 32 chunks).
//
// Terms: three of every fp32 operand.  Two where the result only corrects u or
// is rounded to bf16 would take 308 us instead of 361 for those 64 x 512 tokens
// x 16 heads with their preparation, but the corrections enter the state, which
// then is off by 7e-7 of its norm, 3e-6 with gates near 1 or keys that point one
// way (three: 1.3e-7 and 2.4e-7, as plain fp32), and 3 in 1000 read-outs are not
// the bf16 nearest to the exact one (three: 2 in 10000).
#include "seed_scan_chain.h"

namespace seed {
namespace scan {
namespace {

template <int N>
struct Part {
  static constexpr int value = N;
};

// LDS of one chunk's operands.
template <int RULE, int DK, bool K_Q, bool HAS_M>
struct Stage {
  static constexpr bool DELTA = RULE != kMAMBA2;
  static constexpr int q = kPlane<DK>;
  static constexpr int n = q + (K_Q ? kPlane<DK> : 0);
  static constexpr int m = n + (DELTA ? kTriFrags * 3 * 1024 : 0);
  static constexpr int vec = m + (HAS_M ? kTriFrags * 3 * 1024 : 0);   // P, F, beta
  static constexpr int bytes = vec + 1024;

  // The chunk's loads, PART 0 .. 2 of them (-1: all): spread over the chunk
  // before, so that no wave waits for a full queue.
  template <int W, int PART>
  static __device__ __forceinline__ void load(const ScanArgs& a, uint32_t to, const bf16_t* K,
                                              const bf16_t* Q, uint32_t ld, size_t unit, int rows,
                                              bool transposed, int w) {
    constexpr size_t pack = kTriFrags * 3 * kFrag;
    if (PART <= 0) async_rows<DK, W>(K, Q, ld, rows, to, to + q, K_Q, w);
    if (PART < 0 || PART == 1) {
      if (DELTA)
        async_pack<W>(reinterpret_cast<const uint16_t*>(a.ws + (transposed ? a.at.nt_pack : a.at.n_pack)) +
                              unit * pack, to + n, w);
    }
    if (PART < 0 || PART == 2) {
      if (HAS_M)
        async_pack<W>(reinterpret_cast<const uint16_t*>(a.ws + a.at.m_pack) + unit * pack, to + m, w);
      if (w == W - 1) async_copy(a.ws + a.at.vec + unit * 1024, lane_id() * 16, to + vec);
    }
  }
};

// kSave keeps each chunk's incoming state and E for the backward pass and
// writes no read-outs; kCarry keeps what a segment makes of zero and of the
// unit matrix.
template <int RULE, int DK, int NW, int MODE>
__global__ __launch_bounds__(64 * NW) void chain_forward_kernel(ScanArgs a) {
  constexpr bool DELTA = RULE != kMAMBA2, READ = MODE == kRead, SAVE = MODE == kSave, CARRY = MODE == kCarry;
  constexpr int IT = DK / 16;
  using St = Stage<RULE, DK, READ, READ>;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int w = wave_id();
  const Walk<NW> at(a, a.d_v + (CARRY && DELTA ? DK : 0));
  if (at.c0 > at.c1 || (CARRY && at.c1 == at.chunks)) return;   // nothing is behind a last segment
  const uint32_t lds0 = lds_offset(lds), mine0 = lds0 + 2 * St::bytes + 2048 * w;
  const Range rg = at.rg;
  const int c0 = at.c0, c1 = at.c1, base = at.base;
  const bool unit_cols = CARRY && DELTA && at.col0 >= a.d_v;
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * a.d_v;
  const size_t state = ((size_t)at.seq * a.heads + at.head) * DK * a.d_v;
  const uint32_t g = lane_id() >> 4;
  const uint32_t keep_lane = 4 * g * a.d_v + at.col, state_lane = 8 * g * a.d_v + at.col;
  const bf16_t* K = static_cast<const bf16_t*>(a.k) + ((size_t)rg.start * a.key_heads + at.hk) * DK;
  const bf16_t* Q = static_cast<const bf16_t*>(a.q) + ((size_t)rg.start * a.key_heads + at.hk) * DK;
  const size_t vat = ((size_t)rg.start * a.heads + at.head) * a.d_v + at.col0;
  const bf16_t* V = static_cast<const bf16_t*>(a.v) + vat;
  bf16_t* out = static_cast<bf16_t*>(a.o) + vat;

  f32x4 S[IT];
  if (unit_cols) unit_state(at.col - a.d_v, S);
  else if (!CARRY && at.split)
    load_chunk_state(reinterpret_cast<const float*>(a.ws + a.at.start) + at.segment * DK * a.d_v, at.col0, S);
  else load_state(!CARRY && a.S0 ? a.S0 + state : nullptr, a.d_v, state_lane, S);
  float through = 1.f;

  char* mine = lds + 2 * St::bytes + 2048 * w;   // the wave's columns of V, then of O
  auto values = [&](int c) {
    if (!unit_cols)
      wave_load(V + (size_t)c * kC * vld, vld, min(kC, rg.len - c * kC), mine0);
  };
  if (c0 < c1) {
    St::template load<NW, -1>(a, lds0 + (c0 & 1) * St::bytes, K + (size_t)c0 * kC * kld,
                              Q + (size_t)c0 * kC * kld, kld, (size_t)(base + c0) * a.heads + at.head,
                              min(kC, rg.len - c0 * kC), false, w);
    values(c0);
    async_wait();
    __syncthreads();
  }
  for (int c = c0; c < c1; ++c) {
    const int n = min(kC, rg.len - c * kC);
    const size_t unit = (size_t)(base + c) * a.heads + at.head;
    const char* now = lds + (c & 1) * St::bytes;
    f32x4 u[4], R[4], O[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      u[m] = unit_cols ? zero4() : wave_tile<bf16_t>(mine, m);
      R[m] = O[m] = zero4();
    }
    drop_rows(u, n);
    auto stage = [&](auto part) {
      if (c + 1 < c1)
        St::template load<NW, decltype(part)::value>(
            a, lds0 + ((c + 1) & 1) * St::bytes, K + (size_t)(c + 1) * kC * kld,
            Q + (size_t)(c + 1) * kC * kld, kld, unit + a.heads, min(kC, rg.len - (c + 1) * kC), false, w);
    };
    stage(Part<0>{});
    if (SAVE)
      keep_chunk_state(reinterpret_cast<float*>(a.ws + a.at.state) + unit * DK * a.d_v, at.col0, S);

    if (DELTA || READ) {
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        const Frag<3> s = split_tiles<3>(S[2 * ks], S[2 * ks + 1]);
        Frag<1> f[4];
        if (DELTA) {
#pragma unroll
          for (int m = 0; m < 4; ++m) f[m] = lds_rows<DK, 1>(now, m, ks);
          mma_tiles(R, f, s);
        }
        if (READ) {
#pragma unroll
          for (int m = 0; m < 4; ++m) f[m] = lds_rows<DK, 1>(now + St::q, m, ks);
          mma_tiles(O, f, s);
        }
      }
    }
    stage(Part<1>{});
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 p = lds_vec(now + St::vec, m);
      if (DELTA) u[m] -= p * R[m];
      O[m] *= p;
    }
    if (DELTA) {
      f32x4 b[4], y[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        b[m] = lds_vec(now + St::vec + 512, m);
        y[m] = zero4();
      }
      const Frag<3> x0 = split_tiles<3>(b[0] * u[0], b[1] * u[1]);
      const Frag<3> x1 = split_tiles<3>(b[2] * u[2], b[3] * u[3]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_pack<3>(now + St::n, lower_frag(m, 0));
      mma_tiles(y, f, x0);
      f32x4 z[2] = {y[2], y[3]};
      const Frag<3> h[2] = {lds_pack<3>(now + St::n, lower_frag(2, 1)),
                            lds_pack<3>(now + St::n, lower_frag(3, 1))};
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
    stage(Part<2>{});
    if (READ) {
      constexpr int NU = DELTA ? 3 : 1;   // V itself is one term
      const Frag<NU> x0 = split_tiles<NU>(u[0], u[1]), x1 = split_tiles<NU>(u[2], u[3]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_pack<3>(now + St::m, lower_frag(m, 0));
      mma_tiles(O, f, x0);
      f32x4 z[2] = {O[2], O[3]};
      const Frag<3> h[2] = {lds_pack<3>(now + St::m, lower_frag(2, 1)),
                            lds_pack<3>(now + St::m, lower_frag(3, 1))};
      mma_tiles(z, h, x1);
      O[2] = z[0];
      O[3] = z[1];
      wave_store(out + (size_t)c * kC * vld, vld, n, O, mine);
    }
    if (c + 1 < c1) values(c + 1);
    // S' = P_end S + K^T (F u)
    const float last = *reinterpret_cast<const float*>(now + St::vec + 4 * (kC - 1));
#pragma unroll
    for (int m = 0; m < 4; ++m) u[m] *= lds_vec(now + St::vec + 256, m);
#pragma unroll
    for (int m = 0; m < IT; ++m) S[m] *= last;
    if (CARRY && !DELTA) through *= last;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Frag<3> x = split_tiles<3>(u[2 * ks], u[2 * ks + 1]);
      Frag<1> f[IT];
#pragma unroll
      for (int m = 0; m < IT; ++m) f[m] = lds_cols<DK, 1>(now, m, ks);
      mma_tiles(S, f, x);
    }
    async_wait();
    __syncthreads();
  }
  if (READ && c1 == at.chunks) keep_state(a.S + state, a.d_v, state_lane, S);
  if (CARRY) {
    float* trans = reinterpret_cast<float*>(a.ws + a.at.trans);
    if (unit_cols) keep_chunk_state(trans + at.segment * DK * DK, at.col0 - a.d_v, S);
    else keep_chunk_state(reinterpret_cast<float*>(a.ws + a.at.carry) + at.segment * DK * a.d_v, at.col0, S);
    if (!DELTA && threadIdx.x == 0) trans[at.segment] = through;
  }
}

// The chunks from the last to the first, H the gradient of the state behind
// the chunk.  Keeps H and (delta rules) Y, writes dV and dS0.
// (LOCAL: from H = 0, keeps only what a segment passes back.)
template <int RULE, int DK, int NW, bool LOCAL>
__global__ __launch_bounds__(64 * NW) void chain_reverse_kernel(ScanArgs a) {
  constexpr bool DELTA = RULE != kMAMBA2;
  constexpr int IT = DK / 16;
  using St = Stage<RULE, DK, true, true>;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int w = wave_id();
  const Walk<NW> at(a, a.d_v);
  if (at.c0 > at.c1 || (LOCAL && at.c0 == 0)) return;   // nothing is before a first segment
  const uint32_t lds0 = lds_offset(lds), mine0 = lds0 + 2 * St::bytes + 2048 * w;
  const Range rg = at.rg;
  const int c0 = at.c0, c1 = at.c1, base = at.base;
  const size_t kld = (size_t)a.key_heads * DK, vld = (size_t)a.heads * a.d_v;
  const size_t state = ((size_t)at.seq * a.heads + at.head) * DK * a.d_v;
  const uint32_t g = lane_id() >> 4;
  const uint32_t keep_lane = 4 * g * a.d_v + at.col, state_lane = 8 * g * a.d_v + at.col;
  const bf16_t* K = static_cast<const bf16_t*>(a.k) + ((size_t)rg.start * a.key_heads + at.hk) * DK;
  const bf16_t* Q = static_cast<const bf16_t*>(a.q) + ((size_t)rg.start * a.key_heads + at.hk) * DK;
  const size_t vat = ((size_t)rg.start * a.heads + at.head) * a.d_v + at.col0;
  const bf16_t* dO = static_cast<const bf16_t*>(a.dO) + vat;
  bf16_t* dV = static_cast<bf16_t*>(a.dv) + vat;

  f32x4 H[IT];
  // in the segments' own first pass the last one starts from dS
  if (at.split && !LOCAL)
    load_chunk_state(reinterpret_cast<const float*>(a.ws + a.at.start) + at.segment * DK * a.d_v, at.col0, H);
  else load_state(c1 == at.chunks && a.dS ? a.dS + state : nullptr, a.d_v, state_lane, H);

  char* mine = lds + 2 * St::bytes + 2048 * w;   // the wave's columns of dO, then of dV
  if (c0 < c1) {
    const int c = c1 - 1, rows = min(kC, rg.len - c * kC);
    St::template load<NW, -1>(a, lds0 + (c & 1) * St::bytes, K + (size_t)c * kC * kld,
                          Q + (size_t)c * kC * kld, kld, (size_t)(base + c) * a.heads + at.head, rows,
                          true, w);
    wave_load(dO + (size_t)c * kC * vld, vld, rows, mine0);
    async_wait();
    __syncthreads();
  }
  for (int c = c1 - 1; c >= c0; --c) {
    const int n = min(kC, rg.len - c * kC);
    const size_t unit = (size_t)(base + c) * a.heads + at.head;
    const char* now = lds + (c & 1) * St::bytes;
    auto stage = [&](auto part) {
      if (c > c0)
        St::template load<NW, decltype(part)::value>(
            a, lds0 + ((c - 1) & 1) * St::bytes, K + (size_t)(c - 1) * kC * kld,
            Q + (size_t)(c - 1) * kC * kld, kld, unit - a.heads, kC, true, w);
    };
    stage(Part<0>{});
    if (!LOCAL)
      keep_chunk_state(reinterpret_cast<float*>(a.ws + a.at.grad) + unit * DK * a.d_v, at.col0, H);

    // dU = F (K H) + M^T dO
    f32x4 y[4], go[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      y[m] = zero4();
      go[m] = wave_tile<bf16_t>(mine, m);
    }
    drop_rows(go, n);
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      const Frag<3> h = split_tiles<3>(H[2 * ks], H[2 * ks + 1]);
      Frag<1> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_rows<DK, 1>(now, m, ks);
      mma_tiles(y, f, h);
    }
    stage(Part<1>{});
#pragma unroll
    for (int m = 0; m < 4; ++m) y[m] *= lds_vec(now + St::vec + 256, m);
    {
      const Frag<1> x0 = split_tiles<1>(go[0], go[1]), x1 = split_tiles<1>(go[2], go[3]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_pack<3>(now + St::m, upper_frag(m, 1));
      mma_tiles(y, f, x1);
      f32x4 z[2] = {y[0], y[1]};
      const Frag<3> h[2] = {lds_pack<3>(now + St::m, upper_frag(0, 0)),
                            lds_pack<3>(now + St::m, upper_frag(1, 0))};
      mma_tiles(z, h, x0);
      y[0] = z[0];
      y[1] = z[1];
    }
    if (DELTA) {
      f32x4 b[4], t[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        b[m] = lds_vec(now + St::vec + 512, m);
        t[m] = zero4();
      }
      const Frag<3> x0 = split_tiles<3>(b[0] * y[0], b[1] * y[1]);
      const Frag<3> x1 = split_tiles<3>(b[2] * y[2], b[3] * y[3]);
      Frag<3> f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = lds_pack<3>(now + St::n, upper_frag(m, 1));
      mma_tiles(t, f, x1);
      f32x4 z[2] = {t[0], t[1]};
      const Frag<3> h[2] = {lds_pack<3>(now + St::n, upper_frag(0, 0)),
                            lds_pack<3>(now + St::n, upper_frag(1, 0))};
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
    stage(Part<2>{});
    if (!LOCAL) wave_store(dV + (size_t)c * kC * vld, vld, n, y, mine);
    if (c > c0) wave_load(dO + (size_t)(c - 1) * kC * vld, vld, kC, mine0);

    // dS = P_end H + Q^T (P dO) - K^T (P dR)
    const float last = *reinterpret_cast<const float*>(now + St::vec + 4 * (kC - 1));
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 p = lds_vec(now + St::vec, m);
      go[m] *= p;
      y[m] *= -p;
    }
#pragma unroll
    for (int m = 0; m < IT; ++m) H[m] *= last;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Frag<3> x = split_tiles<3>(go[2 * ks], go[2 * ks + 1]);
      Frag<1> f[IT];
#pragma unroll
      for (int m = 0; m < IT; ++m) f[m] = lds_cols<DK, 1>(now + St::q, m, ks);
      mma_tiles(H, f, x);
      if (DELTA) {
        const Frag<3> z = split_tiles<3>(y[2 * ks], y[2 * ks + 1]);
#pragma unroll
        for (int m = 0; m < IT; ++m) f[m] = lds_cols<DK, 1>(now, m, ks);
        mma_tiles(H, f, z);
      }
    }
    async_wait();
    __syncthreads();
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

template <int RULE, int DK, int NW>
hipError_t chain(const ScanArgs& a, int what, hipStream_t stream) {
  constexpr size_t own = 2048 * NW;
  constexpr size_t read = 2 * Stage<RULE, DK, true, true>::bytes + own;
  constexpr size_t save = 2 * Stage<RULE, DK, false, false>::bytes + own;
  constexpr size_t back = 2 * Stage<RULE, DK, true, true>::bytes + own;
  static_assert(read <= 160 * 1024 && save <= 160 * 1024 && back <= 160 * 1024, "LDS of a CU");
  // (segments are walked by four waves: walk_waves)
  if constexpr (NW == 4) {
    if (what == 3)
      return launch(chain_forward_kernel<RULE, DK, NW, kCarry>, a, a.d_v + (RULE != kMAMBA2 ? DK : 0), NW, save, stream);
    if (what == 4) return launch(chain_reverse_kernel<RULE, DK, NW, true>, a, a.d_v, NW, back, stream);
  }
  switch (what) {
    case 0: return launch(chain_forward_kernel<RULE, DK, NW, kRead>, a, a.d_v, NW, read, stream);
    case 1: return launch(chain_forward_kernel<RULE, DK, NW, kSave>, a, a.d_v, NW, save, stream);
    case 2: return launch(chain_reverse_kernel<RULE, DK, NW, false>, a, a.d_v, NW, back, stream);
    default: return hipErrorInvalidValue;
  }
}
template <int RULE>
hipError_t chain_shape(const ScanArgs& a, int what, hipStream_t stream) {
  if (a.d_k == 64) return chain<RULE, 64, 4>(a, what, stream);
  return walk_waves(a) == 4 ? chain<RULE, 128, 4>(a, what, stream)
                            : chain<RULE, 128, 8>(a, what, stream);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_chain(const ScanArgs& a, int what, hipStream_t stream) {
  return a.rule == kGDN ? scan::chain_shape<kGDN>(a, what, stream)
                        : scan::chain_shape<kMAMBA2>(a, what, stream);
}

}  // namespace seed
