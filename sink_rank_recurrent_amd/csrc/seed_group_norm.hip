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
// Bound by HBM: a team of lanes keeps a group in registers, so each input is
// read once and each output written once; the statistics are two passes over
// the registers.  Teams are 16 to 256 threads, by the group's width, so that
// a thread holds one to four 16-byte vectors of 16-bit values (32 single
// values where d is no multiple of 8).
#include "seed_device.h"
#include "seed_sequence_launch.h"

namespace seed {
namespace {

constexpr int kThreads = 256;

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
    else *p = (bf16_t)round_nearest16<kStoreBF16>(x[0]);
  } else if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[j] = round_nearest16<kStoreBF16>(x[2 * j]) | (round_nearest16<kStoreBF16>(x[2 * j + 1]) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }
__device__ __forceinline__ float act_of(int act, float x) {
  const float s = sigmoid(x);
  return act == kActNone ? x : act == kActSilu ? x * s : s;
}
// act(x) and its derivative
__device__ __forceinline__ void act_both(int act, float x, float& y, float& d) {
  const float s = sigmoid(x);
  y = act == kActNone ? x : act == kActSilu ? x * s : s;
  d = act == kActNone ? 1.f : act == kActSilu ? s * (1.f + x * (1.f - s)) : s * (1.f - s);
}

// Sum over a team of LG threads, the same bits in each of them.
template <int LG>
__device__ __forceinline__ float team_sum(float x, float* lds) {
#pragma unroll
  for (int m = 1; m < (LG < 64 ? LG : 64); m *= 2) x += __shfl_xor(x, m);
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

// Where a team's item lies: the weights' group and the first value of x.
struct Item {
  size_t at;
  bool live;
};

template <int LG, int NV, int VW, typename XT, typename IT>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a, long long items) {
  __shared__ float lds[kThreads / 64];
  constexpr int TEAMS = kThreads / LG;
  const int lane = threadIdx.x % LG;
  const long long item = (long long)blockIdx.x * TEAMS + threadIdx.x / LG;
  if (LG <= 64 && item >= items) return;   // a whole block shares its item otherwise
  const size_t at = (size_t)item * a.d;
  const XT* X = static_cast<const XT*>(a.x) + at;
  const IT* Z = static_cast<const IT*>(a.gate) + at;
  const size_t wat = a.weight_groups == 1 ? 0 : (size_t)(item % a.groups) * a.d;
  const float inv = 1.f / (float)a.d;

  float h[NV][VW], z[NV][VW];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * LG + lane) * VW;
#pragma unroll
    for (int j = 0; j < VW; ++j) h[v][j] = z[v][j] = 0.f;
    if (c < a.d) {
      load_values<VW>(X + c, h[v]);
      if (a.gate) load_values<VW>(Z + c, z[v]);
    }
  }
  if (a.gate) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        z[v][j] = act_of(a.act, z[v][j]);
        if (a.gate_first) h[v][j] *= z[v][j];
      }
  }
  float mean = 0.f;
  if (a.centered) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) mean += (v * LG + lane) * VW < a.d ? h[v][j] : 0.f;
    mean = team_sum<LG>(mean, lds) * inv;
  }
  float var = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      h[v][j] -= mean;
      var += (v * LG + lane) * VW < a.d ? h[v][j] * h[v][j] : 0.f;
    }
  var = team_sum<LG>(var, lds) * inv;
  const float rstd = 1.f / sqrtf(var + a.eps);

  IT* Yp = static_cast<IT*>(a.y) + at;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * LG + lane) * VW;
    if (c >= a.d) continue;
    float w[VW], b[VW], y[VW];
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      w[j] = 1.f;
      b[j] = 0.f;
    }
    if (a.weight) load_values<VW>(a.weight + wat + c, w);
    if (a.bias) load_values<VW>(a.bias + wat + c, b);
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      const float n = h[v][j] * rstd * w[j] + b[j];
      y[j] = !a.gate ? act_of(a.act, n) : a.gate_first ? n : n * z[v][j];
    }
    store_values<VW>(Yp + c, y);
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

  for (long long first = (long long)blockIdx.x * TEAMS; first < items;
       first += (long long)gridDim.x * TEAMS) {
    const long long item = first + team;
    if (LG <= 64 && item >= items) break;
    const size_t at = (split ? (size_t)item * a.groups + blockIdx.y : (size_t)item) * a.d;
    const XT* X = static_cast<const XT*>(a.x) + at;
    const IT* Z = static_cast<const IT*>(a.gate) + at;
    const IT* DY = static_cast<const IT*>(a.dy) + at;
    float x[NV][VW], z[NV][VW], g[NV][VW];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LG + lane) * VW;
#pragma unroll
      for (int j = 0; j < VW; ++j) x[v][j] = z[v][j] = g[v][j] = 0.f;
      if (c < a.d) {
        load_values<VW>(X + c, x[v]);
        load_values<VW>(DY + c, g[v]);
        if (a.gate) load_values<VW>(Z + c, z[v]);
      }
    }
    // h in place of x (gate first: x is needed again, with act(z) beside it)
    float h[NV][VW], mean = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        h[v][j] = a.gate && a.gate_first ? x[v][j] * act_of(a.act, z[v][j]) : x[v][j];
        mean += (v * LG + lane) * VW < a.d ? h[v][j] : 0.f;
      }
    mean = a.centered ? team_sum<LG>(mean, lds) * inv : 0.f;
    float var = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        h[v][j] -= mean;
        var += (v * LG + lane) * VW < a.d ? h[v][j] * h[v][j] : 0.f;
      }
    const float rstd = 1.f / sqrtf(team_sum<LG>(var, lds) * inv + a.eps);

    // g becomes dhat, h becomes hat
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        const bool in = (v * LG + lane) * VW < a.d;
        const float hat = h[v][j] * rstd, n = hat * w[v][j] + b[v][j];
        float dn = g[v][j], y, d;
        if (!a.gate) {
          act_both(a.act, n, y, d);
          dn *= d;
        } else if (!a.gate_first) {
          act_both(a.act, z[v][j], y, d);
          z[v][j] = dn * n * d;   // the gate's gradient
          dn *= y;
        }
        dw[v][j] += in ? dn * hat : 0.f;
        db[v][j] += in ? dn : 0.f;
        const float dhat = dn * w[v][j];
        g[v][j] = dhat;
        h[v][j] = hat;
        s1 += in ? dhat : 0.f;
        s2 += in ? dhat * hat : 0.f;
      }
    s1 = a.centered ? team_sum<LG>(s1, lds) * inv : 0.f;
    s2 = team_sum<LG>(s2, lds) * inv;
    XT* DX = static_cast<XT*>(a.dx) + at;
    IT* DZ = static_cast<IT*>(a.dgate) + at;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LG + lane) * VW;
      if (c >= a.d) continue;
      float dx[VW];
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        dx[j] = rstd * (g[v][j] - s1 - h[v][j] * s2);
        if (a.gate && a.gate_first) {
          float y, d;
          act_both(a.act, z[v][j], y, d);
          z[v][j] = dx[j] * x[v][j] * d;
          dx[j] *= y;
        }
      }
      store_values<VW>(DX + c, dx);
      if (a.gate) store_values<VW>(DZ + c, z[v]);
    }
  }

  if (!sums) return;
  // the block's part: teams added in order
  float* out = a.ws + ((size_t)blockIdx.x * a.weight_groups + (split ? blockIdx.y : 0)) * 2 * a.d;
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

// dweight and dbias: the parts summed by 16 threads a channel, then those in
// order.
__global__ __launch_bounds__(kThreads) void parts_kernel(NormArgs a) {
  __shared__ float lds[16][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), row = threadIdx.x >> 4;
  const int total = a.weight_groups * 2 * a.d;   // [group][dw, db][d]
  float s = 0.f;
  if (c < total)
    for (int p = row; p < a.parts; p += 16) s += a.ws[(size_t)p * total + c];
  lds[row][threadIdx.x & 15] = s;
  __syncthreads();
  if (row == 0 && c < total) {
    s = 0.f;
    for (int j = 0; j < 16; ++j) s += lds[j][threadIdx.x & 15];
    const int grp = c / (2 * a.d), rest = c % (2 * a.d);
    float* to = rest < a.d ? a.dweight : a.dbias;
    if (to) to[(size_t)grp * a.d + rest % a.d] = s;
  }
}

// A team's width for a group of d channels.
int team_of(int d, bool vectors) {
  if (vectors) return d <= 128 ? 16 : d <= 256 ? 32 : d <= 1024 ? 64 : 256;
  return d <= 64 ? 16 : d <= 1024 ? 64 : 256;
}

template <int LG, int NV, int VW, bool BWD>
hipError_t norm_types(const NormArgs& a, hipStream_t stream) {
  const long long items = a.rows * (BWD && a.weight_groups > 1 ? 1 : a.groups);
  const dim3 grid(BWD ? (unsigned)a.parts : (unsigned)((items + kThreads / LG - 1) / (kThreads / LG)),
                  BWD ? a.weight_groups : 1);
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

// Blocks of the backward pass for each weight group: enough for 2048 in
// all, and no more than there are batches of items.
int group_norm_parts(long long rows, int groups, int d, int weight_groups) {
  const int teams = kThreads / team_of(d, d % 8 == 0);
  const long long items = rows * (weight_groups > 1 ? 1 : groups);
  const long long batches = (items + teams - 1) / teams;
  const long long most = weight_groups > 1 ? (2048 + weight_groups - 1) / weight_groups : 2048;
  const long long parts = batches < most ? batches : most;
  return (int)(parts < 1 ? 1 : parts);
}

hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream) { return norm<false>(a, stream); }

hipError_t launch_group_norm_backward(const NormArgs& a, hipStream_t stream) {
  hipError_t e = norm<true>(a, stream);
  if (e != hipSuccess || !(a.dweight || a.dbias)) return e;
  const int total = a.weight_groups * 2 * a.d;
  hipLaunchKernelGGL(parts_kernel, dim3((total + 15) / 16), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace seed
