// Short causal convolution of each channel, its backward pass, and its step
// for single tokens.  With K taps, inputs before a sequence from its S0:
//   pre_t = b + sum_j w_j x_{t - (K - 1) + j},   y_t = act(pre_t)
// and backwards, with e_t = dy_t act'(pre_t):
//   dx_t = sum_j w_j e_{t + (K - 1) - j} (+ dS where x_t is kept in S),
//   dw_j = sum_t e_t x_{t - (K - 1) + j},   db = sum_t e_t.
//
// 2 K + 5 operations a value against 4 (bf16) or 8 bytes: memory.  A thread
// keeps VW neighbouring channels and walks a run of tokens with the last K - 1
// inputs in registers, so that inside a run each input is read once; K - 1 rows
// are read again at the run's start (backward also behind its end).  Nothing is
// shared between threads, so nothing goes through LDS.
#include <type_traits>

#include "seed_channels.h"

namespace seed {
namespace channels {
namespace {

constexpr int kThreads = 256;
// Tokens whose loads are on their way together: whole turns of the window of K
// inputs, so that an input stays in its registers until it has left.
template <int K>
constexpr int kRows = K == 3 ? 6 : 8;
template <int K>
constexpr int kBackRows = K == 3 ? 6 : 4;

// Weights of a thread's channels, tap by tap.
template <int K, int VW>
__device__ __forceinline__ void load_weights(const ConvArgs& a, int c, float (&w)[K][VW], float (&b)[VW]) {
  float t[VW * K];
  const float* p = a.weight + (size_t)c * K;
#pragma unroll
  for (int i = 0; i < VW * K; ++i) t[i] = p[i];
#pragma unroll
  for (int v = 0; v < VW; ++v) {
    b[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][v] = t[v * K + j];
  }
}

template <typename T>
__device__ __forceinline__ const T* row_of(const Rows& r, long long t) {
  return static_cast<const T*>(r.p) + t * r.stride;
}
template <typename T>
__device__ __forceinline__ T* row_of(const OutRows& r, long long t) {
  return static_cast<T*>(r.p) + t * r.stride;
}

// The K - 1 inputs before token t0 of run r: x, S0 or zero.
template <int K, int VW, typename T>
__device__ __forceinline__ void inputs_before(const ConvArgs& a, const Run& r, int c, Packed<VW, T> (&held)[K - 1]) {
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int t = r.t0 - (K - 1) + i;
    held[i].zero();
    if (t >= r.lo) held[i].load(row_of<T>(a.x, t) + c);
    else if (a.S0)
      held[i].load(static_cast<const T*>(a.S0) + ((size_t)r.seq * (K - 1) + (K - 1 + t - r.lo)) * a.channels + c);
  }
}

// The thread's run: threads side by side along the channels (tx of them), then
// along the runs.
struct Place {
  int c, run;
  bool live;
};
template <int VW>
__device__ __forceinline__ Place place(int channels, int tx, int runs) {
  const int lane = threadIdx.x & (tx - 1), row = threadIdx.x / tx;
  const long long run = (long long)blockIdx.x * (kThreads / tx) + row;
  Place p;
  p.c = ((int)blockIdx.y * tx + lane) * VW;
  p.run = run < runs ? (int)run : runs - 1;
  p.live = p.c < channels && run < runs;
  return p;
}
// Its tokens: the wave looks for the sequence of its first thread's run; runs
// of a wave follow each other.  ONE: the wave has one run (64 threads or more
// along the channels), so that what depends on it is scalar.
template <bool ONE>
__device__ __forceinline__ Run tokens_of(const Batch& b, int run) {
  const int first = __builtin_amdgcn_readfirstlane(run);
  int s = sequence_of(b, first);
  if constexpr (ONE) return run_of(b, s, first);
  while (s + 1 < b.n_seq && first_run(b, s + 1) <= run) ++s;
  return run_of(b, s, run);
}

// 64 x 512 tokens x 2048 channels, bf16, 4 taps, SiLU: 60 us, 4.5 TB/s of the
// 6.1 that a large copy reaches (52 where the memory-side cache still has part of
// the arrays; vector unit 47 %).  33 tokens: 5.6 us of a call of 8, bound by the
// launch and one row's latency.
template <int K, int VW, bool ONE, typename T>
__global__ __launch_bounds__(kThreads) void conv_kernel(ConvArgs a, int shift, int runs, int tx) {
  constexpr int R = kRows<K>;
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, shift);
  const Place at = place<VW>(a.channels, tx, runs);
  const Run r = tokens_of<ONE>(b, at.run);
  if (!at.live || (r.t0 >= r.t1 && !r.first)) return;
  const int c = at.c;
  float w[K][VW], bias[VW], x[K][VW];   // token t0 + i of the run: x[(K - 1 + i) % K]
  load_weights<K, VW>(a, c, w, bias);
  Packed<VW, T> held[K - 1];
  inputs_before<K>(a, r, c, held);
  if (r.first && a.S) {
    // what the sequence leaves: this thread has read S0's inputs (S may lie there)
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int t = r.hi - (K - 1) + i;
      Packed<VW, T> s;
      s.zero();
      if (t >= r.lo) s.load(row_of<T>(a.x, t) + c);
      else {
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
          if (k == K - 1 + t - r.lo) s = held[k];
      }
      s.store(static_cast<T*>(a.S) + ((size_t)r.seq * (K - 1) + i) * a.channels + c);
    }
  }
#pragma unroll
  for (int i = 0; i < K - 1; ++i) held[i].floats(x[i]);
  for (int t = r.t0; t < r.t1; t += R) {
    Packed<VW, T> in[R];
#pragma unroll
    for (int j = 0; j < R; ++j) in[j].load(row_of<T>(a.x, t + j < r.t1 ? t + j : r.t1 - 1) + c);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (t + j >= r.t1) break;
      in[j].floats(x[(K - 1 + j) % K]);
      float y[VW];
#pragma unroll
      for (int v = 0; v < VW; ++v) {
        y[v] = bias[v];
#pragma unroll
        for (int k = 0; k < K; ++k) y[v] += w[k][v] * x[(k + j) % K][v];
      }
      if (a.silu) {
#pragma unroll
        for (int v = 0; v < VW; ++v) y[v] *= sigmoid(y[v]);
      }
      Packed<VW, T> out;
      out.from(y);
      out.store(row_of<T>(a.y, t + j) + c);
    }
  }
}

// A block's threads take kThreads / tx runs at a time and keep their parts of
// the weights' gradients in registers; the block adds them up in order through
// LDS, and sums_kernel the blocks' parts.  The pre-activations are made again:
// 4 x 2048 tokens x 4096 channels, bf16, 4 taps, SiLU: 56 us, 3.6 TB/s (46 where
// the memory-side cache still has the arrays), the vector unit busy 66 %; 1040
// workgroups where registers leave room for 768 at once, so that the second round
// is mostly empty; with the sums' launch 61.
template <int K, int VW, bool ONE, typename T>
__global__ __launch_bounds__(kThreads) void conv_backward_kernel(ConvArgs a, int shift, int runs, int tx) {
  constexpr int R = kBackRows<K>;
  __shared__ float lds[(K + 1) * VW * kThreads];
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, shift);
  const int side = kThreads / tx, step = (int)gridDim.x * side;
  const Place at = place<VW>(a.channels, tx, step);
  const int c = at.c;
  float w[K][VW], bias[VW], dw[K][VW], db[VW];
  if (at.live) load_weights<K, VW>(a, c, w, bias);
#pragma unroll
  for (int v = 0; v < VW; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][v] = 0.f;
  }
  for (int base = 0; base < runs; base += step) {   // the wave's lanes together
    const int run = base + at.run < runs ? base + at.run : runs - 1;
    const Run r = tokens_of<ONE>(b, run);
    if (!at.live || base + at.run >= runs || (r.t0 >= r.t1 && !r.first)) continue;
    // token t0 + i of the run: x[(K - 1 + i) % K], and its e likewise
    float x[K][VW], e[K][VW];
    Packed<VW, T> held[K - 1];
    inputs_before<K>(a, r, c, held);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      held[i].floats(x[i]);
#pragma unroll
      for (int v = 0; v < VW; ++v) e[i][v] = 0.f;
    }
    const int end = r.t1 + K - 1;   // the run's last inputs reach K - 1 tokens on
    // R tokens from t on.  PLAIN: all of them in the run, and the K - 1 before
    // them too, so that every one adds to the weights' gradients and has the
    // gradient of an input of the run K - 1 tokens back.
    auto walk = [&](auto plain, int t) {
      constexpr bool PLAIN = decltype(plain)::value;
      Packed<VW, T> in[R], dy[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (!PLAIN) {
          in[j].zero();
          dy[j].zero();
        }
        if (PLAIN || (t + j < r.hi && t + j < end)) {
          in[j].load(row_of<T>(a.x, t + j) + c);
          dy[j].load(row_of<T>(a.dy, t + j) + c);
        }
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int now = t + j, back = now - (K - 1);
        if (!PLAIN && now >= end) break;
        float(&xt)[VW] = x[(K - 1 + j) % K];
        float(&et)[VW] = e[(K - 1 + j) % K];
        float dx[VW];
        in[j].floats(xt);
        dy[j].floats(et);
        if (a.silu) {
#pragma unroll
          for (int v = 0; v < VW; ++v) {
            float pre = bias[v];
#pragma unroll
            for (int k = 0; k < K; ++k) pre += w[k][v] * x[(k + j) % K][v];
            const float s = sigmoid(pre);
            et[v] *= s + pre * s * (1.f - s);
          }
        }
        if (!PLAIN && now >= r.hi) {   // (no token: a NaN of the window would stay in it)
#pragma unroll
          for (int v = 0; v < VW; ++v) et[v] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < VW; ++v) {
          dx[v] = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) dx[v] += w[k][v] * e[(K - 1 - k + j) % K][v];
        }
        if (PLAIN || now < r.t1) {
#pragma unroll
          for (int v = 0; v < VW; ++v) {
            db[v] += et[v];
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][v] += et[v] * x[(k + j) % K][v];
          }
        }
        Packed<VW, T> p;
        if constexpr (PLAIN) {
          p.from(dx);
          p.store(row_of<T>(a.dx, back) + c);
        } else if (back >= r.t0 || r.first) {
          // the gradient of the input K - 1 tokens back: of the run, or of S0
          const int kept = back - (r.hi - (K - 1));   // its place in S
          if (a.dS && kept >= 0) {
            float s[VW];
            p.load(static_cast<const T*>(a.dS) + ((size_t)r.seq * (K - 1) + kept) * a.channels + c);
            p.floats(s);
#pragma unroll
            for (int v = 0; v < VW; ++v) dx[v] += s[v];
          }
          p.from(dx);
          if (back >= r.lo) p.store(row_of<T>(a.dx, back) + c);
          else if (a.dS0)
            p.store(static_cast<T*>(a.dS0) + ((size_t)r.seq * (K - 1) + (K - 1 + back - r.lo)) * a.channels + c);
        }
      }
    };
    for (int t = r.t0; t < end; t += R) {
      if (t - (K - 1) >= r.t0 && t + R <= r.t1) walk(std::true_type{}, t);
      else walk(std::false_type{}, t);
    }
  }
  if (!(a.dweight || a.dbias)) return;
#pragma unroll
  for (int v = 0; v < VW; ++v) {
#pragma unroll
    for (int k = 0; k < K; ++k) lds[(k * VW + v) * kThreads + threadIdx.x] = dw[k][v];
    lds[(K * VW + v) * kThreads + threadIdx.x] = db[v];
  }
  __syncthreads();
  // the block's [K + 1][VW tx] sums, neighbouring channels by neighbouring threads
  const int first = (int)blockIdx.y * tx * VW;
  float* out = a.ws + (size_t)blockIdx.x * (K + 1) * a.channels + first;
  for (int i = threadIdx.x; i < (K + 1) * VW * tx; i += kThreads) {
    const int k = i / (VW * tx), in = i % (VW * tx), lane = in / VW, v = in % VW;
    if (first + in >= a.channels) continue;
    float s = 0.f;
    for (int r = 0; r < side; ++r) s += lds[(k * VW + v) * kThreads + r * tx + lane];
    out[(size_t)k * a.channels + in] = s;
  }
}

// dweight and dbias from the parts [parts][K + 1][channels]: a block sums 64
// channels of one of the K + 1, each of its waves every fourth part, then the
// waves in order.  128 parts of 5 x 4096 (10 MB) in 5 us, with the launch.
__global__ __launch_bounds__(kThreads) void sums_kernel(ConvArgs a, int parts) {
  __shared__ float lds[kThreads];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = blockIdx.y;
  const int c = (int)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < a.channels) {
#pragma unroll 8
    for (int p = wave; p < parts; p += 4) s += a.ws[((size_t)p * (a.width + 1) + k) * a.channels + c];
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (wave != 0 || c >= a.channels) return;
  s = lds[lane] + lds[64 + lane] + lds[128 + lane] + lds[192 + lane];
  if (k < a.width) {
    if (a.dweight) a.dweight[(size_t)c * a.width + k] = s;
  } else if (a.dbias) {
    a.dbias[c] = s;
  }
}

// One token of a sequence: VW channels a thread, all loads on their way
// together.  Bound by the launch where the batch is small (64 x 2048 bf16: 4 us,
// a call 8), by bytes where it is large (256 x 8192 fp32: 12 us, 5.4 TB/s).
template <int K, int VW, typename T>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(ConvArgs a, int tx) {
  const Place at = place<VW>(a.channels, tx, a.n_seq);
  if (!at.live) return;
  const int c = at.c;
  float w[K][VW], bias[VW], x[K][VW], y[VW];
  Packed<VW, T> held[K];
  const size_t state = (size_t)at.run * (K - 1) * a.channels + c;
#pragma unroll
  for (int i = 0; i < K - 1; ++i) held[i].load(static_cast<const T*>(a.S0) + state + (size_t)i * a.channels);
  held[K - 1].load(row_of<T>(a.x, at.run) + c);
  load_weights<K, VW>(a, c, w, bias);
#pragma unroll
  for (int i = 0; i < K; ++i) held[i].floats(x[i]);
#pragma unroll
  for (int v = 0; v < VW; ++v) {
    y[v] = bias[v];
#pragma unroll
    for (int k = 0; k < K; ++k) y[v] += w[k][v] * x[k][v];
    if (a.silu) y[v] *= sigmoid(y[v]);
  }
  Packed<VW, T> out;
  out.from(y);
  out.store(row_of<T>(a.y, at.run) + c);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) held[i + 1].store(static_cast<T*>(a.S) + state + (size_t)i * a.channels);
}

// Threads along the channels: a power of two, at most `most`.
int threads_along(int channels, int vw, int most) {
  const int lanes = (channels + vw - 1) / vw;
  int tx = 1;
  while (tx < lanes && tx < most) tx *= 2;
  return tx;
}
// log2 of a run's tokens: 32, and fewer down to 8 where the runs have fewer
// than 4096 waves, four a SIMD, for `vw` channels a thread (a run of eight
// alone costs nearly what one of sixteen does: 3001 x 2047 single channels
// backward 24 us with runs of 8 or 32, 18 with 16).
constexpr int kLongRun = 5, kShortRun = 3;
int run_shift(int n_seq, int channels, int tokens, int vw) {
  const long long waves = ((long long)channels + 64 * vw - 1) / (64 * vw);
  int shift = kLongRun;
  while (shift > kShortRun && ((long long)(tokens >> shift) + n_seq) * waves < 4096) --shift;
  return shift;
}
int runs_of(int n_seq, int tokens, int shift) { return (tokens >> shift) + n_seq; }

template <int BF16_VECTOR, typename F>
hipError_t with_form(const ConvArgs& a, F f) {
#define SEED_FORM(K)                                                        \
  do {                                                                      \
    if (a.bf16) {                                                           \
      if (a.vectors) f(std::integral_constant<int, K>{}, std::integral_constant<int, BF16_VECTOR>{}, bf16_t{}); \
      else f(std::integral_constant<int, K>{}, std::integral_constant<int, 1>{}, bf16_t{}); \
    } else {                                                                \
      if (a.vectors) f(std::integral_constant<int, K>{}, std::integral_constant<int, 4>{}, float{}); \
      else f(std::integral_constant<int, K>{}, std::integral_constant<int, 1>{}, float{}); \
    }                                                                       \
  } while (0)
  if (a.width == 2) SEED_FORM(2);
  else if (a.width == 3) SEED_FORM(3);
  else SEED_FORM(4);
#undef SEED_FORM
  return hipGetLastError();
}

dim3 grid_of(int runs, int channels, int vw, int tx) {
  const int rows = kThreads / tx, lanes = (channels + vw - 1) / vw;
  return dim3((runs + rows - 1) / rows, (lanes + tx - 1) / tx);
}

}  // namespace
}  // namespace channels

using namespace channels;

// Blocks of the backward pass along the runs: one to a set of runs, 128 at
// most (their sums are read once more).
constexpr int kMostParts = 128;
int parts_of(int runs, int tx) {
  const int sets = (runs + kThreads / tx - 1) / (kThreads / tx);
  return sets < kMostParts ? sets : kMostParts;
}

int short_conv_parts(int n_seq, int channels, int tokens) {
  // whichever form the rows' alignment allows
  int most = 0;
  for (int vw = 1; vw <= 4; vw += 3) {
    const int runs = runs_of(n_seq, tokens, run_shift(n_seq, channels, tokens, vw));
    const int parts = parts_of(runs, threads_along(channels, vw, 64));
    most = parts > most ? parts : most;
  }
  return most;
}

// At most 256 threads for each run and 256 channels, 2^32 in a grid's row.
bool short_conv_fits(int n_seq, int channels, int tokens) {
  return (long long)(tokens >> kLongRun) + n_seq < (1LL << 24) - 1 && (long long)tokens + 64LL < 0x7fffffffLL;
}

hipError_t launch_short_conv(const ConvArgs& a, hipStream_t stream) {
  return with_form<8>(a, [&](auto k, auto vw, auto t) {
    const int shift = run_shift(a.n_seq, a.channels, a.tokens, vw), runs = runs_of(a.n_seq, a.tokens, shift);
    const int tx = threads_along(a.channels, vw, kThreads);
    const dim3 grid = grid_of(runs, a.channels, vw, tx);
    if (tx >= 64) hipLaunchKernelGGL((conv_kernel<k, vw, true, decltype(t)>), grid, dim3(kThreads), 0, stream, a, shift, runs, tx);
    else hipLaunchKernelGGL((conv_kernel<k, vw, false, decltype(t)>), grid, dim3(kThreads), 0, stream, a, shift, runs, tx);
  });
}

hipError_t launch_short_conv_backward(const ConvArgs& a, hipStream_t stream) {
  int parts = 0;
  const hipError_t e = with_form<4>(a, [&](auto k, auto vw, auto t) {
    const int shift = run_shift(a.n_seq, a.channels, a.tokens, vw), runs = runs_of(a.n_seq, a.tokens, shift);
    const int tx = threads_along(a.channels, vw, 64), lanes = (a.channels + vw - 1) / vw;
    parts = parts_of(runs, tx);
    const dim3 grid(parts, (lanes + tx - 1) / tx);
    if (tx >= 64) hipLaunchKernelGGL((conv_backward_kernel<k, vw, true, decltype(t)>), grid, dim3(kThreads), 0, stream, a, shift, runs, tx);
    else hipLaunchKernelGGL((conv_backward_kernel<k, vw, false, decltype(t)>), grid, dim3(kThreads), 0, stream, a, shift, runs, tx);
  });
  if (e != hipSuccess || !(a.dweight || a.dbias)) return e;
  hipLaunchKernelGGL(sums_kernel, dim3((a.channels + 63) / 64, a.width + 1), dim3(kThreads), 0, stream, a, parts);
  return hipGetLastError();
}

hipError_t launch_short_conv_step(const ConvArgs& a, hipStream_t stream) {
  return with_form<8>(a, [&](auto k, auto vw, auto t) {
    const int tx = threads_along(a.channels, vw, kThreads);
    hipLaunchKernelGGL((conv_step_kernel<k, vw, decltype(t)>), grid_of(a.n_seq, a.channels, vw, tx),
                       dim3(kThreads), 0, stream, a, tx);
  });
}

}  // namespace seed
