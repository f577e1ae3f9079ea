// The selective state space scan over sequences (formulas in seed_select.h),
// and its step for single tokens.
#include "seed_select.h"

namespace seed {
namespace channels {
namespace {

// B and C of every token in fp32, [token][group][wave][B of its Q states, C],
// padded with zeros: every block of channels reads them, with aligned vector
// and scalar loads whatever the rows' own strides and type.  Bound by its
// launch: 8192 rows of 2 x 16 in 5 us.
template <typename T>
__global__ __launch_bounds__(kThreads) void prepare_kernel(SelectArgs a) {
  const int Q = a.at.quarter;
  float* out = reinterpret_cast<float*>(a.ws + a.at.rows);
  const size_t total = (size_t)a.tokens * a.groups * 8 * Q, step = (size_t)gridDim.x * kThreads;
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += step) {
    const int in = (int)(i % (8 * Q)), n = in / (2 * Q) * Q + in % Q, what = in / Q & 1;
    const size_t tg = i / (8 * Q), t = tg / a.groups;
    const int g = (int)(tg - t * a.groups);
    float x = 0.f;
    if (n < a.d_state) x = load_scalar(row_of<T>(what ? a.C : a.B, (long long)t) + (size_t)g * a.d_state + n);
    out[i] = x;
  }
}

enum Mode { kWhole = 0, kCarry = 1, kRead = 2 };

// The inputs of a wave's tokens of a tile as they lie in memory.
template <typename T>
struct Raw {
  T x[kOwn], dt[kOwn], z[kOwn];
};
template <typename T>
__device__ __forceinline__ void load_raw(const SelectArgs& a, const Mine& m, int t, int t1, bool gate, Raw<T>& r) {
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    const int at = t + m.wave * kOwn + o, row = at < t1 ? at : t1 - 1;
    const uint32_t in = (uint32_t)m.c * sizeof(T);
    r.x[o] = *in_row<T>(a.x.p, a.x.stride, row, in);
    r.dt[o] = *in_row<T>(a.dt.p, a.dt.stride, row, in);
    if (gate) r.z[o] = *in_row<T>(a.z.p, a.z.stride, row, in);
  }
}

// The sequence that a workgroup's number stands for, long ones first.
// Workgroups start in their numbers' order and go round the CUs, so that each
// CU gets long and short ones alike (24 ragged sequences of 7919 tokens x 4096:
// 149 us, 183 in their own order).  The sequences are ranked among every
// `sets`-th of them, at most 64, by the whole wave.
__device__ __forceinline__ int ranked(const Batch& b, int number) {
  const int sets = (b.n_seq + 63) >> 6, set = number % sets, rank = number / sets;
  const int count = (b.n_seq - set + sets - 1) / sets, lane = (int)__lane_id();
  const int at = set + lane * sets;
  const int len = lane < count ? first_token(b, at + 1) - first_token(b, at) : 0;
  int longer = 0;
  for (int s = 0; s < count; ++s) {
    const int other = __builtin_amdgcn_readlane(len, s);
    longer += other > len || (other == len && s < lane);
  }
  // one lane: the ranks are 0 .. count - 1
  return set + __builtin_ctzll(__ballot(lane < count && longer == rank)) * sets;
}

// MODE kWhole: a sequence from its first state to its last; kCarry: what a
// segment leaves of zero, and the sum of its steps; kRead: a segment's
// read-outs from its first state.
//
// Tiles of 8 tokens: each wave makes the steps of two, all read all eight from
// LDS, and each adds up the four waves' read-outs of its two; the loads of two
// tiles are on their way.  One barrier a tile.  Bound by the vector unit's
// issue slots: kWhole, 24 ragged sequences of 7919 tokens x 4096 channels of 16
// states, bf16: 147 us with all launches, the unit busy 86 % of the cycles with
// four-cycle instructions and 99 % with all (1.9 TB/s).  In segments, 16384 x
// 2048, fp32: kCarry 115 us (78 and 94 %), kRead 135 (78 and 90 %), 264 in all.
template <typename T, int Q, int MODE>
__global__ __launch_bounds__(kThreads, 2) void scan_kernel(SelectArgs a) {
  __shared__ float2 prep[2][kTile][64];                           // the power of two of delta, delta x
  __shared__ float part[MODE == kCarry ? 1 : 2][kWaves][kTile][64];
  __shared__ __attribute__((aligned(16))) float rows[2][RowTile<Q>::kFloats];
  const int block = MODE == kWhole ? blockIdx.x : blockIdx.y;
  const Mine m = mine(a, block / a.at.blocks, block % a.at.blocks);
  const int lane = (int)__lane_id(), c = m.c;
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, MODE == kWhole ? 0 : a.at.shift);
  int t0, t1, s = 0;
  if (MODE == kWhole) {
    s = blockIdx.z * gridDim.y + blockIdx.y;
    if (s >= a.n_seq) return;
    if (a.cu) s = ranked(b, s);
    t0 = first_token(b, s);
    t1 = b.cu ? first_token(b, s + 1) : t0 + b.len;
  } else {
    const Run r = run_of(b, sequence_of(b, blockIdx.x), blockIdx.x);
    t0 = r.t0;
    t1 = r.t1;
    if (t0 >= t1) return;
  }
  float A[Q], h[Q];
  load_rates<Q>(a, m, A);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  float* carry = reinterpret_cast<float*>(a.ws + a.at.carry);
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int n = m.wave * Q + i;
    h[i] = 0.f;
    if (MODE == kWhole && a.S0 && n < a.d_state) h[i] = a.S0[state_at(a, s, c) + n];
    // (a padding state's carry is not a first state: join leaves it as it is)
    if (MODE == kRead && n < a.d_state) h[i] = carry[carry_at<Q>(a, blockIdx.x, n, c)];
  }
  float gone = 0.f;
  const bool gate = MODE != kCarry && a.z.p != nullptr;
  Raw<T> raw, next;
  float x[kOwn], z[kOwn];
  // the tile's steps into LDS; tokens behind the last: steps of zero
  auto prepare = [&](int t, float2 (&to)[kTile][64]) {
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      const int j = m.wave * kOwn + o;
      const bool there = t + j < t1;
      x[o] = load_scalar(&raw.x[o]);
      if (gate) z[o] = load_scalar(&raw.z[o]);
      const float delta = step_of(load_scalar(&raw.dt[o]) + bias, a.softplus), power = in_powers_of_two(delta);
      to[j][lane] = there ? make_float2(power, delta * x[o]) : make_float2(0.f, 0.f);
      if (MODE == kCarry && there) gone += power;
    }
  };
  RowTile<Q> row;
  if (t0 < t1) {
    load_raw(a, m, t0, t1, gate, raw);
    row.load(m.group, t0, t1);
    prepare(t0, prep[0]);
    row.store(rows[0]);
    load_raw(a, m, t0 + kTile, t1, gate, raw);
    row.load(m.group, t0 + kTile, t1);
    __syncthreads();
  }
  take_rates(A);
  int turn = 0;
  for (int t = t0; t < t1; t += kTile, turn ^= 1) {
    load_raw(a, m, t + 2 * kTile, t1, gate, next);
    RowTile<Q> next_row;
    next_row.load(m.group, t + 2 * kTile, t1);
    const ReadOuts<Q> read_outs(m, t, t1);
    // on their way while the steps come from LDS (Q = 16: when they are used)
    float C[Q <= 8 ? kTile : 1][Q];
    if constexpr (MODE != kCarry && Q <= 8) {
#pragma unroll
      for (int j = 0; j < kTile; ++j)
#pragma unroll
        for (int i = 0; i < Q; ++i) C[j][i] = read_outs[j][i];
      next_token();
    }
    float xs[kOwn], zs[kOwn];
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      xs[o] = x[o];
      zs[o] = z[o];
    }
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const float2 k = prep[turn][j][lane];
      Outer<Q, 0> B;
      B.load(rows[turn], m, j);
#pragma unroll
      for (int i = 0; i < Q; ++i) h[i] *= exp2_fast(k.x * A[i]);
      add_outer(h, B, k.y);
      if (MODE != kCarry) {
        const ScalarRow late = read_outs[j];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < Q; ++i) s += (Q <= 8 ? C[Q <= 8 ? j : 0][i] : late[i]) * h[i];
        part[turn][m.wave][j][lane] = s;
      }
    }
    prepare(t + kTile, prep[turn ^ 1]);
    row.store(rows[turn ^ 1]);
    raw = next;
    row = next_row;
    __syncthreads();
    if (MODE == kCarry || !m.live) continue;
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      const int j = m.wave * kOwn + o;
      if (t + j >= t1) continue;
      float y[1] = {D * xs[o]};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) y[0] += part[turn][w][j][lane];
      if (gate) y[0] *= zs[o] * sigmoid(zs[o]);
      Packed<1, T> out;
      out.from(y);
      out.store(in_row<T>(a.y.p, a.y.stride, t + j, (uint32_t)c * sizeof(T)));
    }
  }
  if (MODE == kCarry) {
    // the sum of the steps: each wave has that of its tokens
    prep[0][m.wave][lane].x = gone;   // (every wave is through with it)
    __syncthreads();
    if (m.wave == 0 && m.live)
      reinterpret_cast<float*>(a.ws + a.at.gone)[(size_t)blockIdx.x * a.channels + c] =
          (prep[0][0][lane].x + prep[0][1][lane].x) + (prep[0][2][lane].x + prep[0][3][lane].x);
  }
  if (!m.live || MODE == kRead) return;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int n = m.wave * Q + i;
    if (MODE == kCarry) carry[carry_at<Q>(a, blockIdx.x, n, c)] = h[i];
    else if (n < a.d_state) a.S[state_at(a, s, c) + n] = h[i];
  }
}

// What a segment passes back to its first state, G = a_t (G + ds_t C_t) from its
// last token on, for a state of a channel: one token after the other.
template <typename T>
__device__ __forceinline__ float passed_back(ArgsAgain a, int c, int n, float A, int t0, int t1) {
  const int Q = a->at.quarter, group = c / (a->channels / a->groups);
  const float bias = a->dt_bias ? a->dt_bias[c] : 0.f;
  const float* rows = reinterpret_cast<const float*>(a->ws + a->at.rows) + n / Q * (2 * Q) + Q + n % Q;
  const uint32_t in = (uint32_t)c * sizeof(T);
  float G = 0.f;
#pragma unroll 1
  for (int t = t1 - 1; t >= t0; --t) {
    const float delta = step_of(load_scalar(in_row<T>(a->dt.p, a->dt.stride, t, in)) + bias, a->softplus);
    float ds = load_scalar(in_row<T>(a->dy.p, a->dy.stride, t, in));
    if (a->z.p) {
      const float z = load_scalar(in_row<T>(a->z.p, a->z.stride, t, in));
      ds *= z * sigmoid(z);
    }
    G = exp2_fast(in_powers_of_two(delta) * A) * (G + ds * rows[((size_t)t * a->groups + group) * (8 * Q)]);
  }
  return G;
}

// Whether states of n's wave and c's block overflowed, by segment.
struct Overflow {
  const int* found;
  size_t across;
  __device__ __forceinline__ Overflow(ArgsAgain a, int c, int n) : across((size_t)a->groups * a->at.blocks * kWaves) {
    const int each = a->channels / a->groups, block = c / each * a->at.blocks + c % each / 64;
    found = reinterpret_cast<const int*>(a->ws + a->at.overflow) + (size_t)block * kWaves + n / a->at.quarter;
  }
  __device__ __forceinline__ bool operator[](int at) const { return found[at * across] != 0; }
};

// Tokens t0 .. t1 of segment `at` (tiles from `tile` on) in a join with states
// that grow: the state (or gradient) h before it is left in its place, that
// behind it returned.  Backwards, where the product of decays overflowed within
// the segment (seldom, and slow): what it passes back is made again, and the
// states before its tiles get their part of h here, which is left as zero.
template <bool BACK>
__device__ __forceinline__ float join_grown(ArgsAgain a, int c, int n, float A, int at, size_t tile, int t0, int t1,
                                            bool reverse, bool overflow, float h) {
  const size_t channels = a->channels, row = 4 * a->at.quarter * channels, own = n * channels + c;
  const float* gone = reinterpret_cast<const float*>(a->ws + a->at.gone) + c;
  float* made = reinterpret_cast<float*>(a->ws + (reverse ? a->at.back : a->at.carry)) + at * row + own;
  float x = *made;
  *made = h;
  if (BACK && overflow && reverse) {
    if (!finite(x)) x = a->bf16 ? passed_back<bf16_t>(a, c, n, A, t0, t1) : passed_back<float>(a, c, n, A, t0, t1);
  } else if (BACK && overflow) {
    float* kept = reinterpret_cast<float*>(a->ws + a->at.kept) + tile * row + own;
    const float* before = reinterpret_cast<const float*>(a->ws + a->at.before) + tile * channels + c;
#pragma unroll 1
    for (int t = t0; t < t1; t += kTile, kept += row, before += channels) *kept = grown(A * *before, h, *kept);
    *made = 0.f;
  }
  return grown(A * gone[at * channels], h, x);
}

// The segments' first states, h' = exp(A gone) h + carry, in the carries'
// places, and S; backwards also (blockIdx.z's upper half) the gradients at the
// segments' ends, G' = exp(A gone) G + back, in theirs, and dS0.  A thread is a
// state of a channel of a sequence; the values of kAhead segments are on their
// way together.  Bound by latency, its sequence's segments in turn: 64 of one
// sequence of 2048 channels of 16 states in 12 us, 4 x 16 of 4096 backward in 19
// (17 without the way for states that grow, which takes scalar registers; eight
// waves a SIMD, with six 22).
constexpr int kAhead = 8;
template <bool BACK>
__global__ __launch_bounds__(kThreads, 8) void join_kernel(SelectArgs a) {
  const int c = (int)blockIdx.x * kThreads + threadIdx.x, n = blockIdx.y, NP = 4 * a.at.quarter;
  if (c >= a.channels) return;
  const Batch b = batch_of(a.cu, a.n_seq, a.tokens, a.at.shift);
  float A[1] = {a.A[(size_t)c * a.d_state + n]};
  const bool reverse = BACK && blockIdx.z >= gridDim.z / 2;
  const size_t row = (size_t)NP * a.channels;
  for (int s = reverse ? blockIdx.z - gridDim.z / 2 : blockIdx.z; s < a.n_seq; s += BACK ? gridDim.z / 2 : gridDim.z) {
    const int first = first_run(b, s), lo = first_token(b, s);
    const int end = b.cu ? first_token(b, s + 1) : lo + b.len;
    const int len = end > lo ? end - lo : 0, runs = (len + (1 << a.at.shift) - 1) >> a.at.shift;
    const size_t user = state_at(a, s, c) + n;
    const int from = reverse ? first + runs - 1 : first, way = reverse ? -1 : 1;
    float* made = reinterpret_cast<float*>(a.ws + (reverse ? a.at.back : a.at.carry)) + (size_t)n * a.channels + c;
    const float* gone = reinterpret_cast<const float*>(a.ws + a.at.gone) + c;
    const float* given = reverse ? a.dS : a.S0;
    float h = given ? given[user] : 0.f;
    for (int r = 0; r < runs; r += kAhead) {
      float g[kAhead], x[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int at = from + way * (r + j < runs ? r + j : runs - 1);
        g[j] = gone[(size_t)at * a.channels];
        x[j] = made[(size_t)at * row];
      }
      take_rates(A);                    // (here: it has come with the others)
      const float rate = A[0];
      if (__any(may_grow(a, rate))) {
        bool grows = false;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) grows |= rate * g[j] > 127.f;
        if (BACK && may_grow(a, rate)) {
          const Overflow overflow(args_again(), c, n);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) grows |= overflow[from + way * (r + j < runs ? r + j : runs - 1)];
        }
        if (__any(grows)) {
#pragma unroll 1
          for (int j = 0; j < kAhead && r + j < runs; ++j) {
            const int at = from + way * (r + j), t0 = lo + ((at - first) << a.at.shift);
            const int t1 = end - t0 > (1 << a.at.shift) ? t0 + (1 << a.at.shift) : end;
            h = join_grown<BACK>(args_again(), c, n, rate, at, (size_t)(lo >> 3) + s + ((t0 - lo) >> 3), t0, t1, reverse,
                                 BACK && may_grow(a, rate) && Overflow(args_again(), c, n)[at], h);
          }
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (r + j >= runs) break;
        made[(size_t)(from + way * (r + j)) * row] = h;
        h = fmaf(exp2_fast(rate * g[j]), h, x[j]);
      }
    }
    if (reverse) {
      if (a.dS0) a.dS0[user] = h;
    } else if (!BACK) {
      a.S[user] = h;
    }
  }
}

// One token of several sequences: LP lanes share a channel's states, four each
// (VEC: read and written as one vector), and take kRequests of them with all
// loads on their way together, the channel's rates in registers.  Bound by the
// states' bytes: 256 x 8192 channels of 16 in a call of 49 us, 5.8 TB/s (with
// states through the caches 4 us more; four requests 1 more, eight 8); 64 x 4096
// in 11, the kernel 9.
constexpr int kRequests = 2;
template <typename T, int LP, bool VEC>
__global__ __launch_bounds__(kThreads) void step_kernel(SelectArgs a) {
  const int per = kThreads / LP, part = threadIdx.x % LP;
  const int c = (int)blockIdx.x * per + threadIdx.x / LP;
  const int at = c < a.channels ? c : a.channels - 1, g = at / (a.channels / a.groups);
  const int n0 = part * 4, N = a.d_state;
  // States of 32 MB or more go past the caches: until they are read again, at the
  // next token, a model's other layers have filled these.  us for each of 24
  // layers, states to another array: 33.6 MB 15.8 (through the caches 16.5), 134 MB
  // 48.9 (51.4), but 16.8 MB 9.5 (9.5) and 1 MB 3.8 (3.6); in place equal.
  const bool past = (size_t)a.n_seq * a.channels * N * sizeof(float) >= (size_t)32 << 20;
  auto four = [&](const float* p, float (&v)[4]) {
    if constexpr (VEC) {
      load_vec<4>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = n0 + i < N ? p[i] : 0.f;
    }
  };
  float A[4];
  four(a.A + (size_t)at * N + n0, A);
  const float bias = a.dt_bias ? a.dt_bias[at] : 0.f, D = a.D ? a.D[at] : 0.f;
  for (int b0 = (int)blockIdx.y * kRequests; b0 < a.n_seq; b0 += gridDim.y * kRequests) {
    float h[kRequests][4], x[kRequests], dt[kRequests], z[kRequests], B[kRequests][4], C[kRequests][4];
#pragma unroll
    for (int r = 0; r < kRequests; ++r) {
      const int b = b0 + r < a.n_seq ? b0 + r : a.n_seq - 1;
      four(a.S0 + state_at(a, b, at) + n0, h[r]);
      x[r] = load_scalar(row_of<T>(a.x, b) + at);
      dt[r] = load_scalar(row_of<T>(a.dt, b) + at);
      z[r] = a.z.p ? load_scalar(row_of<T>(a.z, b) + at) : 0.f;
      const T *pB = row_of<T>(a.B, b) + (size_t)g * N + n0, *pC = row_of<T>(a.C, b) + (size_t)g * N + n0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        B[r][i] = VEC || n0 + i < N ? load_scalar(pB + i) : 0.f;
        C[r][i] = VEC || n0 + i < N ? load_scalar(pC + i) : 0.f;
      }
    }
    take_rates(A);   // behind the loads' sending, since it waits (before it 51.2 us, 49.5 so)
#pragma unroll
    for (int r = 0; r < kRequests; ++r) {
      const int b = b0 + r;
      if (b >= a.n_seq) break;
      const float delta = step_of(dt[r] + bias, a.softplus), u = delta * x[r], power = in_powers_of_two(delta);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[r][i] = exp2_fast(power * A[i]) * h[r][i] + u * B[r][i];
        s += C[r][i] * h[r][i];
      }
#pragma unroll
      for (int o = 1; o < LP; o *= 2) s += __shfl_xor(s, o);
      if (c >= a.channels) continue;
      float* S = a.S + state_at(a, b, at) + n0;
      if constexpr (VEC) {
        typedef float f32x4 __attribute__((ext_vector_type(4)));
        if (past) __builtin_nontemporal_store(f32x4{h[r][0], h[r][1], h[r][2], h[r][3]}, reinterpret_cast<f32x4*>(S));
        else store_vec<4>(S, h[r]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < N) S[i] = h[r][i];
      }
      if (part != 0) continue;
      float y[1] = {s + D * x[r]};
      if (a.z.p) y[0] *= z[r] * sigmoid(z[r]);
      Packed<1, T> out;
      out.from(y);
      out.store(row_of<T>(a.y, b) + at);
    }
  }
}

int quarter_of(int d_state) { return d_state <= 8 ? 2 : d_state <= 16 ? 4 : d_state <= 32 ? 8 : 16; }
int blocks_of(int channels, int groups) { return (channels / groups + 63) / 64; }

template <typename T, int Q>
hipError_t scan_types(const SelectArgs& a, hipStream_t stream) {
  const unsigned along = (unsigned)(a.groups * a.at.blocks);
  if (a.at.shift < 0) {
    // sequences along y and z, 2^16 - 1 at most along each
    const unsigned y = a.n_seq < 65535 ? a.n_seq : 65535, z = (a.n_seq + y - 1) / y;
    hipLaunchKernelGGL((scan_kernel<T, Q, kWhole>), dim3(along, y, z), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((scan_kernel<T, Q, kCarry>), dim3(a.at.slots, along), dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = launch_select_join(a, false, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((scan_kernel<T, Q, kRead>), dim3(a.at.slots, along), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace channels

using namespace channels;

SelectLayout select_layout(int n_seq, int channels, int groups, int d_state, int tokens, bool backward) {
  SelectLayout l{};
  l.quarter = quarter_of(d_state);
  l.blocks = blocks_of(channels, groups);
  const long long along = (long long)groups * l.blocks;
  // Forward: whole sequences where these are workgroups enough, or short;
  // segments else (two passes, each making every decay).  us, bf16,
  // 4096 channels: 8 x 1024 tokens 224 whole, 267 in segments; 6 x 1024 214 and
  // 210; 4 x 2048 364 and 274; 1 x 128 31 and 32; 1 x 512 96 and 45.
  // Segments of 256 tokens, and shorter ones where that leaves fewer than 2048
  // workgroups: 16384 x 2048 284 (128 tokens 297, 512 341), 4096 x 4096 185 (128
  // tokens 156, 64 162), 512 x 4096 81 (128 tokens 58, 64 45).  The lengths
  // themselves are on the device: one sequence that is much longer than the mean
  // of many is walked from end to end (4096 channels, 8192 tokens and 63 of one
  // each: 1430 us; alone, in segments, 291).
  if (backward) l.shift = kBackShift;
  else if (n_seq * along >= 384 || tokens / n_seq <= 128) l.shift = -1;
  else
    for (l.shift = 8; l.shift > 6 && (tokens >> l.shift) * along < 2048;) --l.shift;
  const size_t NP = (size_t)l.quarter * 4, T = (size_t)tokens, C = (size_t)channels;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  l.rows = take(T * groups * 2 * NP * 4);
  if (l.shift >= 0) {
    l.slots = (tokens >> l.shift) + n_seq;
    l.carry = take(l.slots * NP * C * 4);
    l.gone = take(l.slots * C * 4);
  }
  if (backward) {
    const size_t tiles = (size_t)(tokens >> 3) + n_seq;
    // Blocks of channels that follow each other in a workgroup add up dB and dC
    // before they are written: as many as leave sixteen workgroups a CU, five
    // rounds of those that fit at once (4 x 2048 x 4096: 639 us with one block,
    // 653 with two, 723 with four and less than two rounds).
    l.set = 4;
    while (l.set > 1 && (long long)l.slots * groups * ((l.blocks + l.set - 1) / l.set) < 4096) l.set /= 2;
    l.sets = (l.blocks + l.set - 1) / l.set;
    l.back = take(l.slots * NP * C * 4);
    l.overflow = take((size_t)l.slots * along * kWaves * 4);
    l.kept = take(tiles * NP * C * 4);
    l.before = take(tiles * C * 4);
    l.sums = take(l.sets * T * groups * 2 * NP * 4);
    // a workgroup goes on to further segments where there are many
    l.parts = l.slots < 512 ? l.slots : 512;
    l.weights = take(l.parts * (NP + 2) * C * 4);
  }
  l.bytes = at;
  return l;
}

// Grids: blocks of channels along y, segments of 64 tokens or more along x with
// 256 threads each, 2^32 threads at most; row numbers of a tile ahead are ints.
bool select_fits(int n_seq, int channels, int groups, int d_state, int tokens) {
  return (long long)groups * blocks_of(channels, groups) <= 65535 &&
         (long long)(tokens >> 6) + n_seq < (1LL << 24) && (long long)tokens + 64 <= 0x7fffffffLL;
}

hipError_t launch_select_prepare(const SelectArgs& a, hipStream_t stream) {
  const size_t total = (size_t)a.tokens * a.groups * 8 * a.at.quarter;
  const size_t blocks = (total + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
  if (a.bf16) hipLaunchKernelGGL((prepare_kernel<bf16_t>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((prepare_kernel<float>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_select_join(const SelectArgs& a, bool backward, hipStream_t stream) {
  const int along = a.n_seq < 32767 ? a.n_seq : 32767;
  const dim3 grid((a.channels + kThreads - 1) / kThreads, a.d_state, backward ? 2 * along : along);
  if (backward) hipLaunchKernelGGL((join_kernel<true>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((join_kernel<false>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_select(const SelectArgs& a, hipStream_t stream) {
  if (a.tokens == 0) {   // S = S0
    SelectArgs none = a;
    none.at.shift = 0;
    return launch_select_join(none, false, stream);
  }
  const hipError_t e = launch_select_prepare(a, stream);
  if (e != hipSuccess) return e;
#define SEED_SCAN(T)                                          \
  (a.at.quarter == 2   ? scan_types<T, 2>(a, stream)          \
   : a.at.quarter == 4 ? scan_types<T, 4>(a, stream)          \
   : a.at.quarter == 8 ? scan_types<T, 8>(a, stream)          \
                       : scan_types<T, 16>(a, stream))
  return a.bf16 ? SEED_SCAN(bf16_t) : SEED_SCAN(float);
#undef SEED_SCAN
}

hipError_t launch_select_step(const SelectArgs& a, hipStream_t stream) {
  const int sets = (a.n_seq + kRequests - 1) / kRequests;
#define SEED_STEP(T, LP, VEC)                                                                              \
  hipLaunchKernelGGL((step_kernel<T, LP, VEC>),                                                            \
                     dim3((a.channels + kThreads / LP - 1) / (kThreads / LP), sets < 65535 ? sets : 65535), \
                     dim3(kThreads), 0, stream, a)
  // whole vectors: 4, 8, 16, 32 or 64 states
#define SEED_STEPS(T)                               \
  do {                                              \
    if (a.d_state == 4) SEED_STEP(T, 1, true);      \
    else if (a.d_state == 8) SEED_STEP(T, 2, true); \
    else if (a.d_state == 16) SEED_STEP(T, 4, true); \
    else if (a.d_state == 32) SEED_STEP(T, 8, true); \
    else if (a.d_state == 64) SEED_STEP(T, 16, true); \
    else if (a.d_state <= 4) SEED_STEP(T, 1, false); \
    else if (a.d_state <= 8) SEED_STEP(T, 2, false); \
    else if (a.d_state <= 16) SEED_STEP(T, 4, false); \
    else if (a.d_state <= 32) SEED_STEP(T, 8, false); \
    else SEED_STEP(T, 16, false);                   \
  } while (0)
  if (a.bf16) SEED_STEPS(bf16_t);
  else SEED_STEPS(float);
#undef SEED_STEPS
#undef SEED_STEP
  return hipGetLastError();
}

}  // namespace seed
