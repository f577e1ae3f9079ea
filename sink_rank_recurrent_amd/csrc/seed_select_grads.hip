// The backward pass of the selective state space scan (formulas in
// seed_select.h), in segments of 64 tokens:
//   ends_kernel   what a segment leaves of zero, h, and what it passes back to
//                 its first state from its own read-outs, sum over t of
//                 (a_1 .. a_t) ds_t C_t, in one walk that makes each decay once
//   join          the segments' first states and the gradients at their ends
//   grads_kernel  each segment forward, keeping the state before every 8th
//                 token in LDS, then 8 tokens at a time backward: their states
//                 and decays again into registers, and the chain rule
//   sums          dB and dC over blocks of channels, dA, dD and ddt_bias over
//                 segments, in a fixed order.
#include "seed_select.h"

namespace seed {
namespace channels {
namespace {

constexpr int kThreads = 64 * kWaves;
constexpr int kShift = 6, kLen = 1 << kShift, kK = kTile, kParts = kLen / kK;

// A token's inputs for a lane: delta, u = delta x, and the gradient of s.
struct Token {
  float x, v, delta, u, z, dy, ds;
};
template <typename T>
__device__ __forceinline__ Token token_of(const SelectArgs& a, int t, int c, float bias, bool live) {
  Token k;
  k.x = load_scalar(row_of<T>(a.x, t) + c);
  k.v = load_scalar(row_of<T>(a.dt, t) + c) + bias;
  k.dy = load_scalar(row_of<T>(a.dy, t) + c);
  k.z = a.z.p ? load_scalar(row_of<T>(a.z, t) + c) : 0.f;
  k.delta = live ? Step{k.v}.of(a.softplus) : 0.f;
  k.u = live ? k.delta * k.x : 0.f;
  k.ds = !live ? 0.f : a.z.p ? k.dy * k.z * sigmoid(k.z) : k.dy;
  return k;
}

template <typename T, int SB>
__global__ __launch_bounds__(kThreads) void ends_kernel(SelectArgs a) {
  const Mine m = mine<SB>(a, blockIdx.y);
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, kShift);
  const int slot = blockIdx.x, c = m.c;
  const Run r = run_of(b, sequence_of(b, slot), slot);
  if (r.t0 >= r.t1) return;
  float A[kStates], h[kStates], P[kStates], G[kStates];
  load_rates<SB>(a, m, A);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
#pragma unroll
  for (int i = 0; i < kStates; ++i) {
    h[i] = G[i] = 0.f;
    P[i] = 1.f;
  }
  float gone = 0.f;
  for (int t = r.t0; t < r.t1; ++t) {
    const Token k = token_of<T>(a, t, c, bias, true);
    const ScalarRow B = row_bc<SB>(a, m, t), C = B + SB * kStates;
    gone += k.delta;
#pragma unroll
    for (int i = 0; i < kStates; ++i) {
      const float d = exp2_fast(k.delta * A[i]);
      h[i] = d * h[i] + k.u * B[i];
      P[i] *= d;
      G[i] += P[i] * (k.ds * C[i]);
    }
  }
  if (!m.live) return;
  float* carry = reinterpret_cast<float*>(a.ws + a.at.carry);
  float* back = reinterpret_cast<float*>(a.ws + a.at.back);
#pragma unroll
  for (int i = 0; i < kStates; ++i) {
    const size_t at = carry_at<SB>(a, slot, m.sb * kStates + i, c);
    carry[at] = h[i];
    back[at] = G[i];
  }
  if (m.sb == 0) reinterpret_cast<float*>(a.ws + a.at.gone)[(size_t)slot * a.channels + c] = gone;
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
    return keep + dpp_mov<ctrl>(give);
  }
}
// Sums over the 64 lanes of 64 values: lane l gets that of value l.
__device__ __forceinline__ float fold64(float (&v)[64]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = fold<5>(v[i], v[i + 32]);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = fold<4>(v[i], v[i + 16]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fold<3>(v[i], v[i + 8]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fold<2>(v[i], v[i + 4]);
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = fold<1>(v[i], v[i + 2]);
  return fold<0>(v[0], v[1]);
}

template <typename T, int SB>
__global__ __launch_bounds__(kThreads) void grads_kernel(SelectArgs a) {
  __shared__ float kept[kWaves][kParts - 1][kStates][64];   // states before each part but the first
  __shared__ float sums[2][kWaves][kK * 2 * kStates];       // dB and dC of 8 tokens, by wave
  __shared__ float part[SB > 1 ? kWaves * 3 * kK * 64 : 1];
  const Mine m = mine<SB>(a, blockIdx.y);
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, kShift);
  const int lane = (int)__lane_id(), wave = threadIdx.x >> 6, c = m.c;
  float A[kStates], dA[kStates];
  load_rates<SB>(a, m, A);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  float dD = 0.f, dbias = 0.f;
#pragma unroll
  for (int i = 0; i < kStates; ++i) dA[i] = 0.f;
  const float* starts = reinterpret_cast<const float*>(a.ws + a.at.carry);
  const float* ends = reinterpret_cast<const float*>(a.ws + a.at.back);
  int turn = 0;

  for (int slot = blockIdx.x; slot < a.at.slots; slot += gridDim.x) {
    const Run r = run_of(b, sequence_of(b, slot), slot);
    if (r.t0 >= r.t1) continue;   // the whole workgroup
    const int parts = (r.t1 - r.t0 + kK - 1) / kK;
    float h[kStates], G[kStates];
#pragma unroll
    for (int i = 0; i < kStates; ++i) {
      const int n = m.sb * kStates + i;
      const size_t at = carry_at<SB>(a, slot, n, c);
      // (join leaves the padding states' carries as they are)
      h[i] = n < a.d_state ? starts[at] : 0.f;
      G[i] = n < a.d_state ? ends[at] : 0.f;
    }
    for (int p = 0; p + 1 < parts; ++p) {
      for (int j = 0; j < kK; ++j) {
        const int t = r.t0 + p * kK + j;
        const Token k = token_of<T>(a, t, c, bias, true);
        const ScalarRow B = row_bc<SB>(a, m, t);
#pragma unroll
        for (int i = 0; i < kStates; ++i) h[i] = exp2_fast(k.delta * A[i]) * h[i] + k.u * B[i];
      }
#pragma unroll
      for (int i = 0; i < kStates; ++i) kept[wave][p][i][lane] = h[i];
    }
    for (int p = parts - 1; p >= 0; --p) {
      const int t0 = r.t0 + p * kK;
      float first[kStates], hs[kK][kStates], d[kK][kStates];
      Token k[kK];
#pragma unroll
      for (int i = 0; i < kStates; ++i) {
        const int n = m.sb * kStates + i;
        first[i] = p > 0 ? kept[wave][p - 1][i][lane] : n < a.d_state ? starts[carry_at<SB>(a, slot, n, c)] : 0.f;
      }
      // tokens behind the segment's last: steps and gradients of zero
#pragma unroll
      for (int j = 0; j < kK; ++j) {
        const int t = t0 + j < r.t1 ? t0 + j : r.t1 - 1;
        k[j] = token_of<T>(a, t, c, bias, t0 + j < r.t1);
        const ScalarRow B = row_bc<SB>(a, m, t);
#pragma unroll
        for (int i = 0; i < kStates; ++i) {
          d[j][i] = exp2_fast(k[j].delta * A[i]);
          hs[j][i] = d[j][i] * (j ? hs[j ? j - 1 : 0][i] : first[i]) + k[j].u * B[i];
        }
      }
      float s[kK], du[kK], rate[kK], total[kK / 2];
#pragma unroll
      for (int jj = kK / 2 - 1; jj >= 0; --jj) {
        float v[64];   // of two tokens: dB, dC
#pragma unroll
        for (int jo = 1; jo >= 0; --jo) {
          const int j = 2 * jj + jo, t = t0 + j < r.t1 ? t0 + j : r.t1 - 1;
          const ScalarRow B = row_bc<SB>(a, m, t), C = B + SB * kStates;
          s[j] = du[j] = rate[j] = 0.f;
#pragma unroll
          for (int i = 0; i < kStates; ++i) {
            G[i] += k[j].ds * C[i];
            v[jo * 32 + i] = m.live ? G[i] * k[j].u : 0.f;
            v[jo * 32 + 16 + i] = m.live ? k[j].ds * hs[j][i] : 0.f;
            s[j] += C[i] * hs[j][i];
            du[j] += G[i] * B[i];
            G[i] *= d[j][i];
            const float q = G[i] * (j ? hs[j ? j - 1 : 0][i] : first[i]);
            rate[j] += A[i] * q;
            dA[i] += k[j].delta * q;
          }
        }
        total[jj] = fold64(v);
      }
      if constexpr (SB > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kK; ++j) {
          part[((wave * kK + j) * 3 + 0) * 64 + lane] = s[j];
          part[((wave * kK + j) * 3 + 1) * 64 + lane] = du[j];
          part[((wave * kK + j) * 3 + 2) * 64 + lane] = rate[j];
        }
        __syncthreads();
        if (m.sb == 0) {
#pragma unroll
          for (int j = 0; j < kK; ++j)
#pragma unroll
            for (int o = 1; o < SB; ++o) {
              s[j] += part[(((wave + o) * kK + j) * 3 + 0) * 64 + lane];
              du[j] += part[(((wave + o) * kK + j) * 3 + 1) * 64 + lane];
              rate[j] += part[(((wave + o) * kK + j) * 3 + 2) * 64 + lane];
            }
        }
      }
      if (m.sb == 0 && m.live) {
#pragma unroll
        for (int j = 0; j < kK; ++j) {
          const int t = t0 + j;
          if (t >= r.t1) continue;
          const float ddelta = k[j].x * du[j] + rate[j] * kLn2;
          const float dv = ddelta * Step{k[j].v}.slope(a.softplus);
          dbias += dv;
          dD += k[j].ds * k[j].x;
          Packed<1, T> out;
          float one[1] = {k[j].delta * du[j] + D * k[j].ds};
          out.from(one);
          out.store(row_of<T>(a.dx, t) + c);
          one[0] = dv;
          out.from(one);
          out.store(row_of<T>(a.ddt, t) + c);
          if (a.z.p) {
            const float g = sigmoid(k[j].z), sy = s[j] + D * k[j].x;
            one[0] = k[j].dy * sy * (g + k[j].z * g * (1.f - g));
            out.from(one);
            out.store(row_of<T>(a.dz, t) + c);
          }
        }
      }
      // dB and dC of the part: the waves of the same states add up in order
      float(&mine_sums)[kWaves][kK * 2 * kStates] = sums[turn];
      turn ^= 1;
#pragma unroll
      for (int jj = 0; jj < kK / 2; ++jj) mine_sums[wave][jj * 64 + lane] = total[jj];
      __syncthreads();
      const int j = threadIdx.x / 32, what = threadIdx.x / 16 & 1, n = threadIdx.x & 15;
      if (t0 + j < r.t1) {
        float* out = reinterpret_cast<float*>(a.ws + a.at.sums) +
                     ((((size_t)m.block * a.tokens + t0 + j) * a.groups + m.group) * 2 + what) * (SB * kStates) + n;
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
          float x = 0.f;
#pragma unroll
          for (int w = sb; w < kWaves; w += SB) x += mine_sums[w][threadIdx.x];
          out[sb * kStates] = x;
        }
      }
    }
  }
  if (!m.live) return;
  float* out = reinterpret_cast<float*>(a.ws + a.at.weights) + (size_t)blockIdx.x * (SB * kStates + 2) * a.channels + c;
#pragma unroll
  for (int i = 0; i < kStates; ++i) out[(size_t)(m.sb * kStates + i) * a.channels] = dA[i];
  if (m.sb == 0) {
    out[(size_t)(SB * kStates) * a.channels] = dD;
    out[(size_t)(SB * kStates + 1) * a.channels] = dbias;
  }
}

// dB and dC: the parts of the blocks of channels, in order.
template <typename T>
__global__ __launch_bounds__(kThreads) void rows_kernel(SelectArgs a) {
  const int NP = a.at.waves * kStates;
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, 0);
  const float* sums = reinterpret_cast<const float*>(a.ws + a.at.sums);
  const int first = first_token(b, 0), end = b.cu ? first_token(b, a.n_seq) : a.tokens;
  const size_t row = (size_t)a.groups * 2 * NP, step = (size_t)gridDim.x * kThreads;
  for (size_t i = first * row + (size_t)blockIdx.x * kThreads + threadIdx.x; i < end * row; i += step) {
    const int n = (int)(i % NP), what = (int)(i / NP & 1);
    if (n >= a.d_state) continue;
    const size_t tg = i / (2 * NP), t = tg / a.groups;
    const int g = (int)(tg - t * a.groups);
    float x[1] = {0.f};
    for (int k = 0; k < a.at.blocks; ++k) x[0] += sums[(size_t)k * a.tokens * row + i];
    Packed<1, T> out;
    out.from(x);
    out.store(row_of<T>(what ? a.dC : a.dB, (long long)t) + (size_t)g * a.d_state + n);
  }
}

// dA, dD and ddt_bias: the parts [part][state + 2][channel], a wave every
// fourth, then the waves in order.
__global__ __launch_bounds__(kThreads) void weights_kernel(SelectArgs a, int parts) {
  __shared__ float lds[kThreads];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, NP = a.at.waves * kStates;
  const int c = (int)blockIdx.x * 64 + lane, n = blockIdx.y, row = n < a.d_state ? n : NP + (n - a.d_state);
  const float* w = reinterpret_cast<const float*>(a.ws + a.at.weights);
  float s = 0.f;
  if (c < a.channels)
    for (int p = wave; p < parts; p += 4) s += w[((size_t)p * (NP + 2) + row) * a.channels + c];
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
}

template <typename T, int SB>
hipError_t grads_types(const SelectArgs& a, hipStream_t stream) {
  const unsigned along = (unsigned)(a.groups * a.at.blocks);
  hipLaunchKernelGGL((ends_kernel<T, SB>), dim3(a.at.slots, along), dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = launch_select_join(a, true, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((grads_kernel<T, SB>), dim3(a.at.parts, along), dim3(kThreads), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t values = (size_t)a.tokens * a.groups * 2 * SB * kStates, blocks = (values + kThreads - 1) / kThreads;
  hipLaunchKernelGGL((rows_kernel<T>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(kThreads), 0, stream, a);
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
  (a.at.waves == 1   ? grads_types<T, 1>(a, stream)            \
   : a.at.waves == 2 ? grads_types<T, 2>(a, stream)            \
                     : grads_types<T, 4>(a, stream))
    e = a.bf16 ? SEED_GRADS(bf16_t) : SEED_GRADS(float);
#undef SEED_GRADS
  } else {
    e = launch_select_join(a, true, stream);   // dS0 = dS
  }
  if (e != hipSuccess) return e;
  // without tokens there are no parts: zero
  hipLaunchKernelGGL(weights_kernel, dim3((a.channels + 63) / 64, a.d_state + 2), dim3(kThreads), 0, stream, a,
                     a.tokens > 0 ? a.at.parts : 0);
  return hipGetLastError();
}

}  // namespace seed
