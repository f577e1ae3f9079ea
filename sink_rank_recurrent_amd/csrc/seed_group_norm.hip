// Group norm of read-outs with a gate and an activation, channels last, and
// its backward pass.  For one group of d channels, act = SiLU or sigmoid:
//   h = x act(z) (gate first) or x;  hat = (h - mean) rstd  (mean 0 unless
//   centered, rstd = (mean((h - mean)^2) + eps)^-1/2);  n = hat w + b
//   y = n act(z) (gate behind), n (gate first), act(n) (no gate)
// and backwards, with dn the gradient of n:
//   dw = sum dn hat, db = sum dn, dhat = dn w,
//   dh = rstd (dhat - mean(dhat) [centered] - hat mean(dhat hat)).
// Everything between the loads and the stores is fp32.
//
// A team of lanes keeps a group in registers, so each input is read once and
// each output written once; the statistics are two passes over the registers.  Teams are 16 to 256 threads, by the group's width, so that
// a thread holds one to four 16-byte vectors of 16-bit values (32 single
// values where d is no multiple of 8).  bf16 values of 128 channels are bound by
// the arithmetic on them as much as by memory: 32768 x 16 groups take 51 us,
// the VALU issuing 73 % of the time (268 MB of inputs and outputs, 201 of them
// past the memory-side cache, 4.0 TB/s), backwards 8192 x 16 with a gate 31 us,
// the VALU 69 %, and 7 us for the weights' gradients.  4001 x 2 groups of 2047
// float32 values backwards take 66 us, the VALU 37 % (239 MB past the cache, 3.6
// TB/s: single values, rows off every alignment), and 12.
// (Sums over rows of 16 lanes by moves between lanes inside the additions and
// the hardware's root; with exchanges through LDS and an IEEE root and
// division 52, 32 and 73.)
#include "seed_device.h"
#include "seed_sequence_launch.h"

namespace seed {
namespace {

constexpr int kThreads = 256;

// 1 / (1 + 2^(-x log2 e)) by the hardware's exponential and reciprocal (one
// ulp each; the argument's rounding is |x| 2^-24 of the exponential).  With
// the library's expf and a division the arithmetic, not the memory, bounds
// the kernels: 88 us instead of 51 for 32768 x 16 x 128 bf16 values.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
template <int VW, typename T>
__device__ __forceinline__ void load_values(const T* __restrict__ p, float (&x)[VW]) {
  if constexpr (VW == 1) {
    x[0] = load_scalar(p);
  } else if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(u[j] << 16);
      x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
}
template <int VW, typename T>
__device__ __forceinline__ void store_values(T* __restrict__ p, const float (&x)[VW]) {
  if constexpr (VW == 1) {
    if constexpr (sizeof(T) == 4) *p = x[0];
    else *p = (bf16_t)round_pair(x[0], 0.f);
  } else if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = round_pair(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// f(act) for the call's activation, one branch for all of a thread's values.
template <int ACT>
struct Act {
  static __device__ __forceinline__ float of(float x) {
    return ACT == kActNone ? x : ACT == kActSilu ? x * sigmoid(x) : sigmoid(x);
  }
  // act(x) and its derivative
  static __device__ __forceinline__ void both(float x, float& y, float& d) {
    const float s = sigmoid(x);
    y = ACT == kActNone ? x : ACT == kActSilu ? x * s : s;
    d = ACT == kActNone ? 1.f : ACT == kActSilu ? s + y * (1.f - s) : s * (1.f - s);
  }
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == kActSilu) f(Act<kActSilu>{});
  else if (act == kActSigmoid) f(Act<kActSigmoid>{});
  else f(Act<kActNone>{});
}

// x plus the x of the lane N on in its row of 16, around the row's end.
template <int N>
__device__ __forceinline__ float add_turned(float x) {
  return x + __int_as_float(
                 __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + N, 0xf, 0xf, true));
}
// Sum over a team of LG threads, the same bits in each of them.
template <int LG>
__device__ __forceinline__ float team_sum(float x, float* lds) {
  static_assert(LG >= 16, "a team has whole rows of 16 lanes");
  x = add_turned<1>(add_turned<2>(add_turned<4>(add_turned<8>(x))));
#pragma unroll
  for (int m = 16; m < (LG < 64 ? LG : 64); m *= 2) x += __shfl_xor(x, m);
  if constexpr (LG > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int j = 0; j < LG / 64; ++j) x += lds[j];
  }
  return x;
}

// One group's values in a thread, values past the group's end 0.
template <int LG, int NV, int VW, typename T>
__device__ __forceinline__ void load_group(const T* __restrict__ p, int lane, int d,
                                           float (&x)[NV][VW]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * LG + lane) * VW;
#pragma unroll
    for (int j = 0; j < VW; ++j) x[v][j] = 0.f;
    if (c < d) load_values<VW>(p + c, x[v]);
  }
}

// 1 / sqrt(x) to a unit in the last place; x is scaled where the hardware
// would take it for 0.
__device__ __forceinline__ float inverse_root(float x) {
  const bool small = x < 0x1p-100f;
  const float r = __builtin_amdgcn_rsqf(small ? x * 0x1p100f : x);
  return small ? r * 0x1p50f : r;
}

// h minus its mean (if centered), in place, and 1 / sqrt(variance + eps).
// Values past the group's end are 0 before and left out of the variance.
template <int LG, int NV, int VW>
__device__ __forceinline__ float normalise(float (&h)[NV][VW], int lane, const NormArgs& a,
                                           float inv, float* lds) {
  if (a.centered) {
    float mean = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) mean += h[v][j];
    mean = team_sum<LG>(mean, lds) * inv;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if ((v * LG + lane) * VW < a.d) {
#pragma unroll
        for (int j = 0; j < VW; ++j) h[v][j] -= mean;
      }
  }
  float var = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < VW; ++j) var += h[v][j] * h[v][j];
  return inverse_root(team_sum<LG>(var, lds) * inv + a.eps);
}

// A block runs over every gridDim.x-th batch of items of one weight group
// (blockIdx.y; all items where the weights are shared), weight and bias in
// registers (read for every item they are four times the bytes of bf16
// values).
template <int LG, int NV, int VW, typename XT, typename IT>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a, long long items) {
  __shared__ float lds[kThreads / 64];
  constexpr int TEAMS = kThreads / LG;
  const int lane = threadIdx.x % LG;
  const bool split = a.weight_groups > 1;
  const size_t wat = split ? (size_t)blockIdx.y * a.d : 0;
  const size_t step = split ? (size_t)a.groups * a.d : a.d;   // from item to item
  const float inv = 1.f / (float)a.d;
  const XT* X = static_cast<const XT*>(a.x) + wat;
  const IT* Z = static_cast<const IT*>(a.gate) + wat;
  IT* Y = static_cast<IT*>(a.y) + wat;

  float w[NV][VW], b[NV][VW];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * LG + lane) * VW;
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      w[v][j] = 1.f;
      b[v][j] = 0.f;
    }
    if (c < a.d) {
      if (a.weight) load_values<VW>(a.weight + wat + c, w[v]);
      if (a.bias) load_values<VW>(a.bias + wat + c, b[v]);
    }
  }
  const long long stride = (long long)gridDim.x * TEAMS;
  for (long long item = (long long)blockIdx.x * TEAMS + threadIdx.x / LG; item < items;
       item += stride) {   // a team's lanes leave together
    float h[NV][VW], z[NV][VW];
    load_group<LG>(X + item * step, lane, a.d, h);
    if (a.gate) {
      load_group<LG>(Z + item * step, lane, a.d, z);
      with_act(a.act, [&](auto act) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < VW; ++j) z[v][j] = act.of(z[v][j]);
      });
      if (a.gate_first) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < VW; ++j) h[v][j] *= z[v][j];
      }
    }
    const float rstd = normalise<LG>(h, lane, a, inv, lds);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) h[v][j] = h[v][j] * rstd * w[v][j] + b[v][j];
    if (!a.gate) {
      with_act(a.act, [&](auto act) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < VW; ++j) h[v][j] = act.of(h[v][j]);
      });
    } else if (!a.gate_first) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VW; ++j) h[v][j] *= z[v][j];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LG + lane) * VW;
      if (c < a.d) store_values<VW>(Y + item * step + c, h[v]);
    }
  }
}

// A block runs over every gridDim.x-th batch of items of one weight group
// (blockIdx.y; all items where the weights are shared) and keeps its part of
// the weights' gradients in registers; the parts are summed in a fixed order
// by parts_kernel.
template <int LG, int NV, int VW, typename XT, typename IT>
__global__ __launch_bounds__(kThreads) void norm_backward_kernel(NormArgs a, long long items) {
  __shared__ float lds[kThreads / 64];
  __shared__ float part[LG < kThreads ? kThreads * NV * VW : 1];
  constexpr int TEAMS = kThreads / LG;
  const int lane = threadIdx.x % LG, team = threadIdx.x / LG;
  const bool split = a.weight_groups > 1;
  const size_t wat = split ? (size_t)blockIdx.y * a.d : 0;
  const float inv = 1.f / (float)a.d;
  const bool sums = a.dweight || a.dbias;

  float w[NV][VW], b[NV][VW], dw[NV][VW], db[NV][VW];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * LG + lane) * VW;
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      w[v][j] = 1.f;
      b[v][j] = dw[v][j] = db[v][j] = 0.f;
    }
    if (c < a.d) {
      if (a.weight) load_values<VW>(a.weight + wat + c, w[v]);
      if (a.bias) load_values<VW>(a.bias + wat + c, b[v]);
    }
  }

  const size_t step = split ? (size_t)a.groups * a.d : a.d;   // from item to item
  const XT* X = static_cast<const XT*>(a.x) + wat;
  const IT* Z = static_cast<const IT*>(a.gate) + wat;
  const IT* DY = static_cast<const IT*>(a.dy) + wat;
  const long long stride = (long long)gridDim.x * TEAMS;
  long long item = (long long)blockIdx.x * TEAMS + team;
  for (; item < items; item += stride) {   // a team's lanes leave together
    float x[NV][VW], z[NV][VW], g[NV][VW], h[NV][VW];
    load_group<LG>(X + item * step, lane, a.d, x);
    load_group<LG>(DY + item * step, lane, a.d, g);
    if (a.gate) load_group<LG>(Z + item * step, lane, a.d, z);
    // gate first: x is needed again, and act's derivative in place of the gate
    if (a.gate && a.gate_first) {
      with_act(a.act, [&](auto act) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            float y, d;
            act.both(z[v][j], y, d);
            h[v][j] = x[v][j] * y;
            z[v][j] = x[v][j] * d;
            x[v][j] = y;
          }
      });
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VW; ++j) h[v][j] = x[v][j];
    }
    const float rstd = normalise<LG>(h, lane, a, inv, lds);
    // h becomes hat, g the gradient of n; the gate behind: z its gradient
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) h[v][j] *= rstd;
    if (!a.gate) {
      with_act(a.act, [&](auto act) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            float y, d;
            act.both(h[v][j] * w[v][j] + b[v][j], y, d);
            g[v][j] *= d;
          }
      });
    } else if (!a.gate_first) {
      with_act(a.act, [&](auto act) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            float y, d;
            act.both(z[v][j], y, d);
            z[v][j] = g[v][j] * (h[v][j] * w[v][j] + b[v][j]) * d;
            g[v][j] *= y;
          }
      });
    }
    // (values past the group's end: g and h are 0)
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        dw[v][j] += g[v][j] * h[v][j];
        db[v][j] += g[v][j];
        g[v][j] *= w[v][j];
        s1 += g[v][j];
        s2 += g[v][j] * h[v][j];
      }
    s1 = a.centered ? team_sum<LG>(s1, lds) * inv : 0.f;
    s2 = team_sum<LG>(s2, lds) * inv;
    XT* DX = static_cast<XT*>(a.dx) + wat + item * step;
    IT* DZ = static_cast<IT*>(a.dgate) + wat + item * step;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LG + lane) * VW;
      if (c >= a.d) continue;
#pragma unroll
      for (int j = 0; j < VW; ++j) g[v][j] = rstd * (g[v][j] - s1 - h[v][j] * s2);
      if (a.gate && a.gate_first) {
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          z[v][j] *= g[v][j];
          g[v][j] *= x[v][j];
        }
      }
      store_values<VW>(DX + c, g[v]);
      if (a.gate) store_values<VW>(DZ + c, z[v]);
    }
  }

  if (!sums) return;
  // the block's part: teams added in order
  const size_t columns = ((size_t)a.weight_groups * 2 * a.d + 3) & ~(size_t)3;
  float* out = a.ws + blockIdx.x * columns + (split ? (size_t)blockIdx.y * 2 * a.d : 0);
  for (int what = 0; what < 2; ++what) {
    float(&acc)[NV][VW] = what == 0 ? dw : db;
    if constexpr (TEAMS > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VW; ++j)
          part[team * (LG * NV * VW) + (v * LG + lane) * VW + j] = acc[v][j];
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += kThreads) {
        float s = 0.f;
        for (int t = 0; t < TEAMS; ++t) s += part[t * (LG * NV * VW) + c];
        out[(size_t)what * a.d + c] = s;
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * LG + lane) * VW;
        if (c < a.d) store_values<VW>(out + (size_t)what * a.d + c, acc[v]);
      }
    }
  }
}

// dweight and dbias: a block sums four neighbouring columns of the parts
// [parts][stride], thread t the parts t, t + 256, ...; then by halves.  Wide
// weights have more columns than a grid has blocks for (2^32 threads along
// x): a block then goes on to the columns a grid further.
constexpr int kPartsBlocks = 1 << 16;
__global__ __launch_bounds__(kThreads) void parts_kernel(NormArgs a) {
  __shared__ float4 lds[kThreads];
  const int total = a.weight_groups * 2 * a.d, stride = (total + 3) & ~3;   // [group][dw, db][d]
  for (int c = blockIdx.x * 4; c < total; c += gridDim.x * 4) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = threadIdx.x; p < a.parts; p += kThreads) {
      const float4 x = *reinterpret_cast<const float4*>(a.ws + (size_t)p * stride + c);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    __syncthreads();   // the columns before are written out
    lds[threadIdx.x] = s;
    for (int half = kThreads / 2; half > 0; half >>= 1) {
      __syncthreads();
      if ((int)threadIdx.x < half) {
        const float4 x = lds[threadIdx.x + half];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        lds[threadIdx.x] = s;
      }
    }
    __syncthreads();
    if (threadIdx.x < 4 && c + (int)threadIdx.x < total) {
      const int at = c + threadIdx.x, grp = at / (2 * a.d), rest = at % (2 * a.d);
      float* to = rest < a.d ? a.dweight : a.dbias;
      if (to) to[(size_t)grp * a.d + rest % a.d] = reinterpret_cast<const float*>(lds)[threadIdx.x];
    }
  }
}

// A team's width for a group of d channels.
int team_of(int d, bool vectors) {
  if (vectors) return d <= 128 ? 16 : d <= 256 ? 32 : d <= 1024 ? 64 : 256;
  return d <= 64 ? 16 : d <= 1024 ? 64 : 256;
}

template <int LG, int NV, int VW, bool BWD>
hipError_t norm_types(const NormArgs& a, hipStream_t stream) {
  const long long items = a.rows * (a.weight_groups > 1 ? 1 : a.groups);
  const dim3 grid((unsigned)a.parts, a.weight_groups);
#define SEED_NORM(XT, IT)                                                                      \
  do {                                                                                         \
    if (BWD)                                                                                   \
      hipLaunchKernelGGL((norm_backward_kernel<LG, NV, VW, XT, IT>), grid, dim3(kThreads), 0,  \
                         stream, a, items);                                                    \
    else                                                                                       \
      hipLaunchKernelGGL((norm_kernel<LG, NV, VW, XT, IT>), grid, dim3(kThreads), 0, stream, a, \
                         items);                                                               \
  } while (0)
  if (a.x_bf16) {
    if (a.io_bf16) SEED_NORM(bf16_t, bf16_t);
    else SEED_NORM(bf16_t, float);
  } else {
    if (a.io_bf16) SEED_NORM(float, bf16_t);
    else SEED_NORM(float, float);
  }
#undef SEED_NORM
  return hipGetLastError();
}

template <bool BWD>
hipError_t norm(const NormArgs& a, hipStream_t stream) {
  const int d = a.d;
  if (d % 8 == 0) {
    if (d <= 128) return norm_types<16, 1, 8, BWD>(a, stream);
    if (d <= 256) return norm_types<32, 1, 8, BWD>(a, stream);
    if (d <= 512) return norm_types<64, 1, 8, BWD>(a, stream);
    if (d <= 1024) return norm_types<64, 2, 8, BWD>(a, stream);
    if (d <= 2048) return norm_types<256, 1, 8, BWD>(a, stream);
    if (d <= 4096) return norm_types<256, 2, 8, BWD>(a, stream);
    return norm_types<256, 4, 8, BWD>(a, stream);
  }
  if (d <= 64) return norm_types<16, 4, 1, BWD>(a, stream);
  if (d <= 256) return norm_types<64, 4, 1, BWD>(a, stream);
  if (d <= 1024) return norm_types<64, 16, 1, BWD>(a, stream);
  if (d <= 2048) return norm_types<256, 8, 1, BWD>(a, stream);
  return norm_types<256, 32, 1, BWD>(a, stream);
}

}  // namespace

// Blocks of the backward pass for each weight group, no more than there are
// batches of items: 2048 in all fill the CUs, but each writes its sums once,
// so fewer, down to 512, where a block has less than some 40 items (8002
// groups of 2047 values: the sums took 39 us of 109 with 2048 blocks).
int group_norm_parts(long long rows, int groups, int d, int weight_groups) {
  const int teams = kThreads / team_of(d, d % 8 == 0);
  const long long items = rows * (weight_groups > 1 ? 1 : groups);
  const long long batches = (items + teams - 1) / teams;
  long long all = rows * groups / 40;
  all = all > 2048 ? 2048 : all < 512 ? 512 : all;
  const long long most = (all + weight_groups - 1) / weight_groups;
  const long long parts = batches < most ? batches : most;
  return (int)(parts < 1 ? 1 : parts);
}

hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream) {
  // 4096 blocks in all, or one for each batch of items
  const int teams = kThreads / team_of(a.d, a.d % 8 == 0);
  const long long items = a.rows * (a.weight_groups > 1 ? 1 : a.groups);
  const long long batches = (items + teams - 1) / teams, most = (4096 + a.weight_groups - 1) / a.weight_groups;
  NormArgs b = a;
  b.parts = (int)(batches < most ? batches : most);
  return norm<false>(b, stream);
}

hipError_t launch_group_norm_backward(const NormArgs& a, hipStream_t stream) {
  hipError_t e = norm<true>(a, stream);
  if (e != hipSuccess || !(a.dweight || a.dbias)) return e;
  const int blocks = (a.weight_groups * 2 * a.d + 3) / 4;
  hipLaunchKernelGGL(parts_kernel, dim3(blocks < kPartsBlocks ? blocks : kPartsBlocks), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace seed
