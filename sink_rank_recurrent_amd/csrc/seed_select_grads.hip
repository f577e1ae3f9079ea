// The backward pass of the selective state space scan (formulas in
// seed_select.h), in segments of 128 tokens:
//   ends_kernel   what a segment leaves of zero, h, and what it passes back to
//                 its first state from its own read-outs, sum over t of
//                 (a_1 .. a_t) ds_t C_t, in one walk that makes each decay
//                 once; the state it has come to before every 8th token
//   join          the segments' first states and the gradients at their ends
//   grads_kernel  8 tokens at a time, the last first: the states and decays
//                 from the state before them (what the segment had made of
//                 zero, and the decayed first state), and the chain rule
//   sums_kernel   dB and dC over sets of blocks of channels, dA, dD and
//                 ddt_bias over segments, in a fixed order.
#include "seed_select.h"

namespace seed {
namespace channels {
namespace {

constexpr int kShift = kBackShift, kTiles = (1 << kShift) / kTile;

// The inputs of a wave's tokens of a tile as they lie in memory.
template <typename T, bool GATE>
struct Raw {
  T x[kOwn], dt[kOwn], z[GATE ? kOwn : 1], dy[kOwn];
};
template <typename T, bool GATE>
__device__ __forceinline__ void load_raw(const Mine& m, int t, int t1, Raw<T, GATE>& r) {
  const ArgsAgain a = args_again();
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    const int at = t + m.wave * kOwn + o, row = at < t1 ? at : t1 - 1;
    const uint32_t in = (uint32_t)m.c * sizeof(T);
    r.x[o] = *in_row<T>(a->x.p, a->x.stride, row, in);
    r.dt[o] = *in_row<T>(a->dt.p, a->dt.stride, row, in);
    r.dy[o] = *in_row<T>(a->dy.p, a->dy.stride, row, in);
    if (GATE) r.z[o] = *in_row<T>(a->z.p, a->z.stride, row, in);
  }
}

// A token's values for a lane; behind the last token steps and gradients of
// zero.  BACK: with what the gradients need behind the walk, softplus' slope
// and dy silu'(z).
struct Token {
  float x, delta, ds, slope, dys;
};
template <bool BACK, typename T, bool GATE>
__device__ __forceinline__ void tokens_of(const Raw<T, GATE>& r, float bias, bool softplus, int there,
                                          Token (&k)[kOwn]) {
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    k[o].x = load_scalar(&r.x[o]);
    k[o].delta = load_scalar(&r.dt[o]) + bias;
    k[o].slope = 1.f;
    const float dy = load_scalar(&r.dy[o]);
    k[o].ds = dy;
    if (GATE) {
      const float z = load_scalar(&r.z[o]), g = sigmoid(z), zg = z * g;
      k[o].ds = dy * zg;
      if (BACK) k[o].dys = dy * (g + zg * (1.f - g));
    }
  }
  if (softplus) {
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      float e;
      const float v = k[o].delta;
      k[o].delta = softplus_of(v, e);
      if (BACK) k[o].slope = softplus_slope(v, e);
    }
  }
#pragma unroll
  for (int o = 0; o < kOwn; ++o)
    if (o >= there) k[o].delta = k[o].ds = 0.f;
}
// The power of two of delta, delta x and ds as the waves share them.
struct Shared {
  float2 step[kTile][64];
  float ds[kTile][64];
  __device__ __forceinline__ void put(int j, int lane, const Token& k, bool there) {
    step[j][lane] = there ? make_float2(in_powers_of_two(k.delta), k.delta * k.x) : make_float2(0.f, 0.f);
    ds[j][lane] = there ? k.ds : 0.f;
  }
};

// Number of the 8 tokens from t on among the batch's tiles: like that of a run.
__device__ __forceinline__ size_t tile_number(const Run& r, int t) { return (size_t)(r.lo >> 3) + r.seq + ((t - r.lo) >> 3); }

// Tiles of 8 tokens as in the forward pass.  The decays' product P goes with
// the states, so that both directions' ends come out of one walk with one
// exponential a state.  P starts at two: where it does not overflow, 2^(A gone)
// does not either, with a power of two between for the roundings; where it does,
// what is passed back is infinite or NaN from there on, which the join finds
// marked.  Bound by the vector unit: 4 x 2048 tokens x 4096 channels of 16 states,
// bf16, in 163 us, busy 87 % with four-cycle instructions, 98 % with all.
template <typename T, int Q, bool GATE>
__global__ __launch_bounds__(kThreads, Q <= 4 ? 4 : Q <= 8 ? 2 : 1) void ends_kernel(SelectArgs a) {
  __shared__ Shared prep[2];
  __shared__ __attribute__((aligned(16))) float rows[2][RowTile<Q>::kFloats];
  const Mine m = mine(a, blockIdx.y / a.at.blocks, blockIdx.y % a.at.blocks);
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, kShift);
  const int slot = blockIdx.x, c = m.c, lane = (int)__lane_id();
  const Run r = run_of(b, sequence_of(b, slot), slot);
  if (r.t0 >= r.t1) return;
  float A[Q], h[Q], P[Q], G[Q];
  load_rates<Q>(a, m, A);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  const bool softplus = a.softplus;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    h[i] = G[i] = 0.f;
    P[i] = 2.f;
  }
  Raw<T, GATE> raw;
  auto prepare = [&](int t, Shared& to) {
    Token k[kOwn];
    const int at = t + m.wave * kOwn;
    tokens_of<false>(raw, bias, softplus, r.t1 - at, k);
#pragma unroll
    for (int o = 0; o < kOwn; ++o) to.put(m.wave * kOwn + o, lane, k[o], at + o < r.t1);
  };
  RowTile<Q> row;
  load_raw(m, r.t0, r.t1, raw);
  row.load(m.group, r.t0, r.t1);
  prepare(r.t0, prep[0]);
  row.store(rows[0]);
  load_raw(m, r.t0 + kTile, r.t1, raw);
  row.load(m.group, r.t0 + kTile, r.t1);
  __syncthreads();
  take_rates(A);
  float gone = 0.f;
  int turn = 0;
  for (int t = r.t0; t < r.t1; t += kTile, turn ^= 1) {
    Raw<T, GATE> next;
    RowTile<Q> next_row;
    load_raw(m, t + 2 * kTile, r.t1, next);
    next_row.load(m.group, t + 2 * kTile, r.t1);
    const size_t tile = tile_number(r, t);
    if (m.live) {
      const ArgsAgain q = args_again();
      const size_t channels = q->channels;
      float* kept = reinterpret_cast<float*>(q->ws + q->at.kept) + (tile * (4 * Q) + m.wave * Q) * channels;
      const uint32_t in = (uint32_t)c * sizeof(float);
#pragma unroll
      for (int i = 0; i < Q; ++i) *in_row<float>(kept, channels, i, in) = h[i];
      if (m.wave == 0)
        *in_row<float>(reinterpret_cast<float*>(q->ws + q->at.before) + tile * channels, 0, 0, in) = gone;
    }
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      if (j > 0 && j % 2 == 0) {
        settle(P);
        settle(G);
        next_token();
      }
      const float2 k = prep[turn].step[j][lane];
      const float ds = prep[turn].ds[j][lane];
      Outer<Q, 0> B;
      Outer<Q, 1> C;
      B.load(rows[turn], m, j);
      C.load(rows[turn], m, j);
      float dsC[Q];
      gone += k.x;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const float d = exp2_fast(k.x * A[i]);
        h[i] *= d;
        P[i] *= d;
        dsC[i] = 0.f;
      }
      add_outer(h, B, k.y);
      add_outer(dsC, C, ds);
#pragma unroll
      for (int i = 0; i < Q; ++i) G[i] += P[i] * dsC[i];
    }
    prepare(t + kTile, prep[turn ^ 1]);
    row.store(rows[turn ^ 1]);
    raw = next;
    row = next_row;
    __syncthreads();
  }
  bool over = false, may = false;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    G[i] *= 0.5f;
    over |= !finite(G[i]);
    may |= may_grow(a, A[i]);
  }
  if (__any(may)) {
    const bool any = __any(over);
    if (lane == 0)
      reinterpret_cast<int*>(a.ws + a.at.overflow)[((size_t)slot * gridDim.y + blockIdx.y) * kWaves + m.wave] = any;
  }
  if (!m.live) return;
  float* carry = reinterpret_cast<float*>(a.ws + a.at.carry);
  float* back = reinterpret_cast<float*>(a.ws + a.at.back);
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const size_t at = carry_at<Q>(a, slot, m.wave * Q + i, c);
    carry[at] = h[i];
    back[at] = G[i];
  }
  if (m.wave == 0) reinterpret_cast<float*>(a.ws + a.at.gone)[(size_t)slot * a.channels + c] = gone;
}

// p + q where the lane's bit is 0: p of both halves of the lanes, where it is
// 1: q of both.  Bits 5 and 4 by the exchanges between rows of 16 lanes, 3 to
// 0 by moves inside the rows (bit 2 by the mirror of 8 lanes).
template <int BIT>
__device__ __forceinline__ float fold(float p, float q) {
  if constexpr (BIT >= 4) {
    const auto r = BIT == 5 ? __builtin_amdgcn_permlane32_swap(__float_as_uint(p), __float_as_uint(q), false, false)
                            : __builtin_amdgcn_permlane16_swap(__float_as_uint(p), __float_as_uint(q), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else {
    const bool high = (__lane_id() >> BIT) & 1;
    const float keep = high ? q : p, give = high ? p : q;
    constexpr int ctrl = BIT == 3 ? 0x128 : BIT == 2 ? 0x141 : BIT == 1 ? 0x4E : 0xB1;
    return keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), ctrl, 0xf, 0xf, true));
  }
}
// Sums over every fourth of the 64 lanes of 16 values: lane l gets that of
// value l / 4 over the lanes l % 4, l % 4 + 4, ...
__device__ __forceinline__ float fold16(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fold<5>(v[i], v[i + 8]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fold<4>(v[i], v[i + 4]);
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = fold<3>(v[i], v[i + 2]);
  return fold<2>(v[0], v[1]);
}

// A set of blocks of channels of one group (blockIdx.y) over every
// gridDim.x-th segment.  A wave keeps 8 tokens' decays and states of a quarter
// in registers (three waves a SIMD), from the kept state before them, so that
// nothing runs backwards through a decay.  Bound by the vector unit: 87
// instructions a token of four states, 46 of them the states' own formulas, 18
// the sums of dB and dC over the lanes, the others the tokens' own (softplus,
// gate, dx, ddt, dz), which the waves share.  4 x 2048 tokens x 4096 channels,
// bf16: 425 us, busy 80 % with four-cycle instructions, 90 % with all.
template <typename T, int Q, bool GATE>
__global__ __launch_bounds__(kThreads, Q <= 4 ? 3 : Q <= 8 ? 2 : 1) void grads_kernel(SelectArgs a) {
  // dB and dC of 8 tokens and a wave's states are summed over the lanes 16
  // values at a time, those of kFoldTile tokens and kFoldStates states each
  constexpr int kFoldTile = Q < 8 ? kTile / Q : 1, kFoldStates = Q < 8 ? Q : 8;
  constexpr int kFolds = Q < 4 ? 1 : Q / 4;               // values a lane has at last
  __shared__ Shared prep;
  __shared__ __attribute__((aligned(16))) float rows[RowTile<Q>::kFloats];
  __shared__ float2 part[kWaves][kTile][64];                        // du and the rates' part of ddelta
  __shared__ float part_s[GATE ? kWaves : 1][kTile][64];            // C.h
  __shared__ float sums[kTiles][kWaves][kFolds][64];
  const int lane = (int)__lane_id();
  const int group = blockIdx.y / a.at.sets, set = blockIdx.y % a.at.sets;
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, kShift);

  for (int slot = blockIdx.x; slot < a.at.slots; slot += gridDim.x) {
    const Run r = run_of(b, sequence_of(b, slot), slot);
    const bool none = r.t0 >= r.t1;   // the whole workgroup
    const int tiles = none ? 0 : (r.t1 - r.t0 + kTile - 1) / kTile;
    const int first_block = set * a.at.set;
    for (int block = first_block; block < (set + 1) * a.at.set && block < a.at.blocks; ++block) {
      const Mine m = mine(a, group, block);
      const int c = m.c;
      float A[Q], dA[Q], H[Q], G[Q];
      load_rates<Q>(a, m, A);
      const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
      float dD = 0.f, dbias = 0.f;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int n = m.wave * Q + i;
        dA[i] = H[i] = G[i] = 0.f;
        if (!none && n < a.d_state) {   // (join leaves the padding states' carries as they are)
          H[i] = reinterpret_cast<const float*>(a.ws + a.at.carry)[carry_at<Q>(a, slot, n, c)];
          G[i] = reinterpret_cast<const float*>(a.ws + a.at.back)[carry_at<Q>(a, slot, n, c)];
        }
      }
      Raw<T, GATE> raw;
      RowTile<Q> row;
      float made[Q], gone;              // before the tile: the segment's own state, its steps
      auto load_tile = [&](int t0) {
        load_raw(m, t0, r.t1, raw);
        row.load(group, t0, r.t1);
        const ArgsAgain q = args_again();
        const size_t tile = tile_number(r, t0), channels = q->channels;
        const float* kept = reinterpret_cast<const float*>(q->ws + q->at.kept) + (tile * (4 * Q) + m.wave * Q) * channels;
        const uint32_t in = (uint32_t)c * sizeof(float);
#pragma unroll
        for (int i = 0; i < Q; ++i) made[i] = *in_row<float>(kept, channels, i, in);
        gone = *in_row<float>(reinterpret_cast<const float*>(q->ws + q->at.before) + tile * channels, 0, 0, in);
      };
      if (!none) load_tile(r.t0 + (tiles - 1) * kTile);
      take_rates(A);
      for (int p = tiles - 1; p >= 0; --p) {
        const int t0 = r.t0 + p * kTile;
        float first[Q], hs[kTile][Q], d[kTile][Q];
#pragma unroll
        for (int i = 0; i < Q; ++i)   // (from 2^127.75 on H is zero, and `made` all of the state)
          first[i] = fmaf(exp2_fast(__builtin_elementwise_minimum(gone * A[i], 127.75f)), H[i], made[i]);
        Token own[kOwn];
        const int at = t0 + m.wave * kOwn;
        tokens_of<true>(raw, bias, args_again()->softplus, r.t1 - at, own);
#pragma unroll
        for (int o = 0; o < kOwn; ++o)   // lanes without a channel add nothing to dB and dC
          prep.put(m.wave * kOwn + o, lane, own[o], at + o < r.t1 && m.live);
        row.store(rows);
        if (p > 0) load_tile(t0 - kTile);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kTile; ++j) {
          if (Q >= 4 && j % 2 == 0) next_token();
          const float2 k = prep.step[j][lane];
          Outer<Q, 0> B;
          B.load(rows, m, j);
#pragma unroll
          for (int i = 0; i < Q; ++i) {
            d[j][i] = exp2_fast(k.x * A[i]);
            hs[j][i] = d[j][i] * (j ? hs[j ? j - 1 : 0][i] : first[i]);
          }
          add_outer(hs[j], B, k.y);
        }
        int again = lane;   // the steps are read a second time: 24 registers less
        asm volatile("" : "+v"(again));
        float sum[Q];     // of 16 values each: the last fold's groups of lanes
#pragma unroll
        for (int f = Q - 1; f >= 0; --f) {
          float v[16];    // dB and dC of 8 / Q tokens, or of half a token's states
          next_token();
#pragma unroll
          for (int jj = kFoldTile - 1; jj >= 0; --jj) {
            const int j = f * kTile / Q + jj, i0 = Q > 8 ? (f & 1) * 8 : 0;
            float B[Q], C[Q];
            row_values<Q, 0>(rows, m, j, B);
            if (GATE) row_values<Q, 1>(rows, m, j, C);
            const float2 k = prep.step[j][again];
            const float ds = prep.ds[j][again];
            if (Q <= 8 || i0 > 0) {
              Outer<Q, 1> outer;
              outer.load(rows, m, j);
              add_outer(G, outer, ds);
            }
            float s = 0.f, du = 0.f, rate = 0.f;
#pragma unroll
            for (int ii = 0; ii < kFoldStates; ++ii) {
              const int i = i0 + ii;
              v[(jj * 2 + 0) * kFoldStates + ii] = G[i] * k.y;
              v[(jj * 2 + 1) * kFoldStates + ii] = ds * hs[j][i];
              if (GATE) s += C[i] * hs[j][i];
              du += G[i] * B[i];
              G[i] *= d[j][i];
              const float q = G[i] * (j ? hs[j ? j - 1 : 0][i] : first[i]);
              rate += A[i] * q;
              dA[i] += k.x * q;
            }
            if (Q > 8 && i0 == 0) {   // the upper half of the token's states came first
              if (GATE) s += part_s[m.wave][j][lane];
              du += part[m.wave][j][lane].x;
              rate += part[m.wave][j][lane].y;
            }
            part[m.wave][j][lane] = make_float2(du, rate);
            if (GATE) part_s[m.wave][j][lane] = s;
          }
          sum[f] = fold16(v);
          settle(G);
          settle(dA);
        }
#pragma unroll
        for (int f = 0; f < kFolds; ++f) {
          float total;
          if constexpr (Q > 2) total = fold<0>(fold<1>(sum[4 * f], sum[4 * f + 2]), fold<1>(sum[4 * f + 1], sum[4 * f + 3]));
          else {
            total = fold<1>(sum[0], sum[1]);
            total += dpp_mov<0xB1>(total);
          }
          float& to = sums[p][m.wave][f][lane];
          to = block == first_block ? total : to + total;
        }
        __syncthreads();
        if (!m.live) continue;
        const ArgsAgain q = args_again();
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
          const int j = m.wave * kOwn + o;
          const int t = t0 + j;
          const uint32_t in = (uint32_t)c * sizeof(T);
          if (t >= r.t1) continue;
          // the read-out's gradient from LDS again (the wave's own)
          const Token& k = own[o];
          const float ds = prep.ds[j][lane];
          float s = 0.f, du = 0.f, rate = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            const float2 v = part[w][j][lane];
            if (GATE) s += part_s[w][j][lane];
            du += v.x;
            rate += v.y;
          }
          const float dv = (k.x * du + rate) * k.slope;
          dbias += dv;
          dD += ds * k.x;
          Packed<1, T> out;
          float one[1] = {k.delta * du + D * ds};
          out.from(one);
          out.store(in_row<T>(q->dx.p, q->dx.stride, t, in));
          one[0] = dv;
          out.from(one);
          out.store(in_row<T>(q->ddt.p, q->ddt.stride, t, in));
          if (GATE) {
            one[0] = (s + D * k.x) * k.dys;
            out.from(one);
            out.store(in_row<T>(q->dz.p, q->dz.stride, t, in));
          }
        }
      }
      // the block's part of the weights' gradients: that of the workgroup's
      // segments before, and this one's
      __syncthreads();
      part[m.wave][0][lane] = make_float2(dD, dbias);
      __syncthreads();
      if (m.live) {
        float* out = reinterpret_cast<float*>(a.ws + a.at.weights) + (size_t)blockIdx.x * (4 * Q + 2) * a.channels + c;
        const bool more = slot >= (int)gridDim.x;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          float& to = out[(size_t)(m.wave * Q + i) * a.channels];
          const float x = dA[i] * kLn2;
          to = more ? to + x : x;
        }
        if (m.wave < 2) {
          float x = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) x += m.wave == 0 ? part[w][0][lane].x : part[w][0][lane].y;
          float& to = out[(size_t)(4 * Q + m.wave) * a.channels];
          to = more ? to + x : x;
        }
      }
    }
    // dB and dC of the set: lane l has value l / 4 of fold 4 f + l % 4 (Q = 2:
    // of fold l / 2 % 2)
    const int wave = (int)threadIdx.x >> 6;
    for (int p = 0; p < tiles; ++p)
#pragma unroll
      for (int f = 0; f < kFolds; ++f) {
        const int fold = Q > 2 ? 4 * f + (lane & 3) : lane >> 1 & 1, value = lane >> 2;
        const int jj = value / (2 * kFoldStates), what = value / kFoldStates & 1;
        const int j = fold * kTile / Q + jj, i = (Q > 8 ? (fold & 1) * 8 : 0) + value % kFoldStates;
        const int t = r.t0 + p * kTile + j;
        if (t < r.t1 && (Q > 2 || (lane & 1) == 0))
          reinterpret_cast<float*>(a.ws + a.at.sums)[((((size_t)set * a.tokens + t) * a.groups + group) * 4 + wave) * (2 * Q) +
                                                     what * Q + i] = sums[p][wave][f][lane];
      }
  }
}

// Sums of the workgroups' parts, two kinds of blocks in one launch.  The first
// `weights` blocks: dA, dD and ddt_bias from the parts [part][states, dD,
// ddt_bias][channel], 64 channels of one of them a block, each of its waves every
// fourth part, then the waves in order.  The others: dB and dC from the parts of
// the sets of channels, in order.  8192 tokens of 2 x 16 from 64 sets (67 MB) and
// 18 x 4096 weights from 68 parts (20 MB) in 18 us, 4.9 TB/s.
template <typename T>
__global__ __launch_bounds__(kThreads) void sums_kernel(SelectArgs a, int parts, int weights) {
  const int Q = a.at.quarter, NP = 4 * Q;
  if ((int)blockIdx.x < weights) {   // the whole block
    __shared__ float lds[kThreads];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, rows = a.d_state + 2;
    const int c = (int)blockIdx.x / rows * 64 + lane, n = (int)blockIdx.x % rows;
    const int row = n < a.d_state ? n : NP + (n - a.d_state);
    const float* w = reinterpret_cast<const float*>(a.ws + a.at.weights);
    float s = 0.f;
    if (c < a.channels) {
#pragma unroll 8
      for (int p = wave; p < parts; p += 4) s += w[((size_t)p * (NP + 2) + row) * a.channels + c];
    }
    lds[threadIdx.x] = s;
    __syncthreads();
    if (wave != 0 || c >= a.channels) return;
    s = lds[lane] + lds[64 + lane] + lds[128 + lane] + lds[192 + lane];
    if (n < a.d_state) a.dA[(size_t)c * a.d_state + n] = s;
    else if (n == a.d_state) {
      if (a.dD) a.dD[c] = s;
    } else if (a.ddt_bias) {
      a.ddt_bias[c] = s;
    }
    return;
  }
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, 0);
  const float* sums = reinterpret_cast<const float*>(a.ws + a.at.sums);
  const int first = first_token(b, 0), end = b.cu ? first_token(b, a.n_seq) : a.tokens;
  const size_t row = (size_t)a.groups * 8 * Q, step = (size_t)(gridDim.x - weights) * kThreads;
  for (size_t i = first * row + (size_t)(blockIdx.x - weights) * kThreads + threadIdx.x; i < end * row; i += step) {
    const int in = (int)(i % (8 * Q)), n = in / (2 * Q) * Q + in % Q, what = in / Q & 1;
    if (n >= a.d_state) continue;
    const size_t tg = i / (8 * Q), t = tg / a.groups;
    const int g = (int)(tg - t * a.groups);
    float x[1] = {0.f};
#pragma unroll 8
    for (int k = 0; k < a.at.sets; ++k) x[0] += sums[(size_t)k * a.tokens * row + i];
    Packed<1, T> out;
    out.from(x);
    out.store(row_of<T>(what ? a.dC : a.dB, (long long)t) + (size_t)g * a.d_state + n);
  }
}

// At most 2^14 blocks of channels by 66.  Without tokens there are no parts: zero.
template <typename T>
hipError_t launch_sums(const SelectArgs& a, hipStream_t stream) {
  const int weights = (a.channels + 63) / 64 * (a.d_state + 2);
  const size_t values = (size_t)a.tokens * a.groups * 8 * a.at.quarter, blocks = (values + kThreads - 1) / kThreads;
  hipLaunchKernelGGL((sums_kernel<T>), dim3((unsigned)(weights + (blocks < 4096 ? blocks : 4096))), dim3(kThreads), 0,
                     stream, a, a.tokens > 0 ? a.at.parts : 0, weights);
  return hipGetLastError();
}

template <typename T, int Q>
hipError_t grads_types(const SelectArgs& a, hipStream_t stream) {
  const dim3 ends(a.at.slots, a.groups * a.at.blocks), grads(a.at.parts, a.groups * a.at.sets);
  if (a.z.p) hipLaunchKernelGGL((ends_kernel<T, Q, true>), ends, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((ends_kernel<T, Q, false>), ends, dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = launch_select_join(a, true, stream);
  if (e != hipSuccess) return e;
  if (a.z.p) hipLaunchKernelGGL((grads_kernel<T, Q, true>), grads, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((grads_kernel<T, Q, false>), grads, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace channels

using namespace channels;

hipError_t launch_select_backward(const SelectArgs& a, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.tokens > 0) {
    e = launch_select_prepare(a, stream);
    if (e != hipSuccess) return e;
#define SEED_GRADS(T)                                          \
  (a.at.quarter == 2   ? grads_types<T, 2>(a, stream)          \
   : a.at.quarter == 4 ? grads_types<T, 4>(a, stream)          \
   : a.at.quarter == 8 ? grads_types<T, 8>(a, stream)          \
                       : grads_types<T, 16>(a, stream))
    e = a.bf16 ? SEED_GRADS(bf16_t) : SEED_GRADS(float);
#undef SEED_GRADS
  } else {
    e = launch_select_join(a, true, stream);   // dS0 = dS
  }
  if (e != hipSuccess) return e;
  return a.bf16 ? launch_sums<bf16_t>(a, stream) : launch_sums<float>(a, stream);
}

}  // namespace seed
