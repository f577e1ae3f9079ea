// C ABI of the operators on channels (declared in include/seed_channels.h):
// host validation, then the launchers.
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/seed_channels.h"
#include "seed_channels_launch.h"
#include "seed_error.h"

namespace {

seed_status fail(seed_status st, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  return seed::set_error(st, text);
}

seed_status ok() { return seed::set_error(SEED_OK, ""); }

seed_status device_status(const char* fn, hipError_t e) {
  if (e != hipSuccess)
    return fail(SEED_E_DEVICE, "%s: HIP error %d (%s)", fn, (int)e, hipGetErrorString(e));
  return ok();
}

constexpr int kMostChannels = 1 << 20;

#define SEED_TRY(call)              \
  do {                              \
    const seed_status s_ = (call);  \
    if (s_ != SEED_OK) return s_;   \
  } while (0)

// An array of a call: `rows` rows of `len` values of `size` bytes, `stride`
// values apart (dense arrays: one row).
struct Array {
  const char* name;
  const void* p;
  size_t rows, len, size;
  long long stride;
  bool must;     // NULL is refused
  size_t align;

  size_t bytes() const {
    return rows == 0 || len == 0 ? 0 : ((rows - 1) * (size_t)stride + len) * size;
  }
};

Array dense(const char* name, const void* p, size_t values, size_t size, bool must) {
  return {name, p, 1, values, size, (long long)values, must, 16};
}

seed_status check_array(const char* fn, const Array& a) {
  if (a.rows == 0 || a.len == 0) return SEED_OK;   // nothing of it is touched
  if (a.p == nullptr)
    return a.must ? fail(SEED_E_ARG, "%s: %s is NULL", fn, a.name) : SEED_OK;
  if ((reinterpret_cast<uintptr_t>(a.p) & (a.align - 1)) != 0)
    return fail(SEED_E_ARG, "%s: %s is not %zu-byte aligned", fn, a.name, a.align);
  if (a.stride < 0 || (size_t)a.stride < a.len)
    return fail(SEED_E_SHAPE, "%s: %s has rows of %zu values, %lld apart", fn, a.name, a.len, a.stride);
  if ((unsigned long long)a.stride > (1ull << 40) || (unsigned long long)a.stride > (1ull << 60) / a.rows)
    return fail(SEED_E_UNSUPPORTED, "%s: rows of %s are more than 2^40 values apart, or reach beyond 2^60", fn,
                a.name);
  return SEED_OK;
}

// Whether two arrays share a byte.  Rows of the same stride are slices of
// one array, side by side; other strided arrays are taken as whole.
bool overlap(const Array& a, const Array& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes() == 0 || b.bytes() == 0) return false;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
  if (p >= q + b.bytes() || q >= p + a.bytes()) return false;
  const size_t step = (size_t)a.stride * a.size;
  if (a.rows > 1 && b.rows > 1 && step == (size_t)b.stride * b.size) {
    const size_t one = a.len * a.size, two = b.len * b.size;
    const size_t at = p <= q ? (q - p) % step : (step - (p - q) % step) % step;   // of b's rows in a's
    return !(at >= one && at + two <= step);
  }
  return true;
}

// Every array by itself, then the outputs against all that is read and each
// other.
template <int NO, int NI>
seed_status check_arrays(const char* fn, const Array (&out)[NO], const Array (&in)[NI]) {
  for (const Array& a : in) SEED_TRY(check_array(fn, a));
  for (const Array& a : out) SEED_TRY(check_array(fn, a));
  for (int i = 0; i < NO; ++i) {
    for (const Array& b : in)
      if (overlap(out[i], b)) return fail(SEED_E_ARG, "%s: %s overlaps %s", fn, out[i].name, b.name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j]))
        return fail(SEED_E_ARG, "%s: %s overlaps %s", fn, out[i].name, out[j].name);
  }
  return SEED_OK;
}

seed_status check_sequences(const char* fn, int n_seq, int channels, int tokens, const int* cu) {
  if (n_seq <= 0 || channels <= 0 || tokens < 0)
    return fail(SEED_E_SHAPE, "%s: n_seq and channels must be positive and tokens at least 0 (got %d, %d, %d)",
                fn, n_seq, channels, tokens);
  if (channels > kMostChannels)
    return fail(SEED_E_UNSUPPORTED, "%s: %d channels, above 2^20", fn, channels);
  if (cu == nullptr && tokens % n_seq != 0)
    return fail(SEED_E_SHAPE, "%s: %d tokens do not make %d equal sequences", fn, tokens, n_seq);
  return SEED_OK;
}

seed_status check_conv(const char* fn, int n_seq, int channels, int width, int tokens, const int* cu,
                       int io_dtype, int activation) {
  SEED_TRY(check_sequences(fn, n_seq, channels, tokens, cu));
  if (width < 2 || width > 4)
    return fail(SEED_E_UNSUPPORTED, "%s: width %d not supported (use 2, 3 or 4)", fn, width);
  if (!seed::short_conv_fits(n_seq, channels, tokens))
    return fail(SEED_E_UNSUPPORTED, "%s: n_seq, tokens or channels exceed the grid limit", fn);
  if (io_dtype != SEED_F32 && io_dtype != SEED_BF16)
    return fail(SEED_E_ARG, "%s: unknown dtype %d", fn, io_dtype);
  if (activation != SEED_ACT_NONE && activation != SEED_ACT_SILU)
    return fail(SEED_E_ARG, "%s: unknown activation %d (use none or SiLU)", fn, activation);
  return SEED_OK;
}

seed::ConvArgs conv_args(int n_seq, int channels, int width, int tokens, const int* cu, const void* x,
                         long long x_stride, int io_dtype, const float* weight, const float* bias,
                         const void* S0, int activation) {
  seed::ConvArgs a{};
  a.n_seq = n_seq;
  a.channels = channels;
  a.width = width;
  a.tokens = tokens;
  a.cu = cu;
  a.bf16 = io_dtype == SEED_BF16;
  a.silu = activation == SEED_ACT_SILU;
  a.x = {x, x_stride};
  a.weight = weight;
  a.bias = bias;
  a.S0 = S0;
  return a;
}

// Rows of whole 16-byte vectors of eight channels.
bool vector_rows(const void* p, long long stride, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride * (long long)size) % 16 == 0;
}

seed_status check_select(const char* fn, int n_seq, int channels, int groups, int d_state, int tokens,
                         const int* cu, int io_dtype) {
  SEED_TRY(check_sequences(fn, n_seq, channels, tokens, cu));
  if (groups <= 0 || channels % groups != 0)
    return fail(SEED_E_SHAPE, "%s: channels (%d) must be a multiple of groups (%d)", fn, channels, groups);
  if (d_state <= 0 || d_state > 64)
    return fail(SEED_E_UNSUPPORTED, "%s: d_state %d not supported (use 1 .. 64)", fn, d_state);
  if (!seed::select_fits(n_seq, channels, groups, d_state, tokens))
    return fail(SEED_E_UNSUPPORTED, "%s: n_seq, tokens, channels or groups exceed the grid limit", fn);
  if (io_dtype != SEED_F32 && io_dtype != SEED_BF16)
    return fail(SEED_E_ARG, "%s: unknown dtype %d", fn, io_dtype);
  return SEED_OK;
}

seed::SelectArgs select_args(int n_seq, int channels, int groups, int d_state, int tokens, const int* cu,
                             const void* x, long long x_stride, const void* dt, long long dt_stride,
                             const float* A, const void* B, long long B_stride, const void* C,
                             long long C_stride, int io_dtype, const float* D, const void* z,
                             long long z_stride, const float* dt_bias, int softplus, const float* S0) {
  seed::SelectArgs a{};
  a.n_seq = n_seq;
  a.channels = channels;
  a.groups = groups;
  a.d_state = d_state;
  a.tokens = tokens;
  a.cu = cu;
  a.bf16 = io_dtype == SEED_BF16;
  a.softplus = softplus != 0;
  a.x = {x, x_stride};
  a.dt = {dt, dt_stride};
  a.B = {B, B_stride};
  a.C = {C, C_stride};
  a.z = {z, z_stride};
  a.A = A;
  a.D = D;
  a.dt_bias = dt_bias;
  a.S0 = S0;
  return a;
}

}  // namespace

extern "C" {

seed_status seed_short_conv(int n_seq, int channels, int width, int tokens, const int* cu_seqlens,
                            const void* x, long long x_stride, int io_dtype, const float* weight,
                            const float* bias, const void* S0, int activation, void* y,
                            long long y_stride, void* S, void* stream) {
  const char* fn = "seed_short_conv";
  SEED_TRY(check_conv(fn, n_seq, channels, width, tokens, cu_seqlens, io_dtype, activation));
  const size_t e = io_dtype == SEED_BF16 ? 2 : 4, T = (size_t)tokens, C = (size_t)channels;
  const size_t state = (size_t)n_seq * (width - 1) * C;
  const Array out[] = {{"y", y, T, C, e, y_stride, true, e}, dense("S", S, state, e, false)};
  Array in[] = {{"x", x, T, C, e, x_stride, true, e},
                dense("weight", weight, C * width, 4, true),
                dense("bias", bias, C, 4, false),
                dense("S0", S0, state, e, false),
                dense("cu_seqlens", cu_seqlens, (size_t)n_seq + 1, 4, false)};
  in[4].align = 4;
  if (S0 != nullptr && S == S0) {   // in place, but checked like the others
    SEED_TRY(check_array(fn, in[3]));
    in[3].p = nullptr;
  }
  SEED_TRY(check_arrays(fn, out, in));
  if (tokens == 0 && S == nullptr) return ok();
  seed::ConvArgs a = conv_args(n_seq, channels, width, tokens, cu_seqlens, x, x_stride, io_dtype, weight,
                               bias, S0, activation);
  a.y = {y, y_stride};
  a.S = S;
  a.vectors = channels % 8 == 0 && vector_rows(x, x_stride, e) && vector_rows(y, y_stride, e);
  return device_status(fn, seed::launch_short_conv(a, static_cast<hipStream_t>(stream)));
}

seed_status seed_short_conv_backward(int n_seq, int channels, int width, int tokens,
                                     const int* cu_seqlens, const void* x, long long x_stride,
                                     int io_dtype, const float* weight, const float* bias,
                                     const void* S0, int activation, const void* dy,
                                     long long dy_stride, const void* dS, void* dx,
                                     long long dx_stride, float* dweight, float* dbias, void* dS0,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "seed_short_conv_backward";
  SEED_TRY(check_conv(fn, n_seq, channels, width, tokens, cu_seqlens, io_dtype, activation));
  const size_t e = io_dtype == SEED_BF16 ? 2 : 4, T = (size_t)tokens, C = (size_t)channels;
  const size_t state = (size_t)n_seq * (width - 1) * C;
  const bool sums = dweight != nullptr || dbias != nullptr;
  const size_t want = sums ? seed_short_conv_workspace_bytes(n_seq, channels, width, tokens) : 0;
  const Array out[] = {{"dx", dx, T, C, e, dx_stride, true, e},
                       dense("dweight", dweight, C * width, 4, false),
                       dense("dbias", dbias, C, 4, false),
                       dense("dS0", dS0, state, e, false),
                       dense("workspace", sums ? workspace : nullptr, want, 1, sums)};
  Array in[] = {{"x", x, T, C, e, x_stride, true, e},
                {"dy", dy, T, C, e, dy_stride, true, e},
                dense("weight", weight, C * width, 4, true),
                dense("bias", bias, C, 4, false),
                dense("S0", S0, state, e, false),
                dense("dS", dS, state, e, false),
                dense("cu_seqlens", cu_seqlens, (size_t)n_seq + 1, 4, false)};
  in[6].align = 4;
  SEED_TRY(check_arrays(fn, out, in));
  if (sums && workspace_bytes < want)
    return fail(SEED_E_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, want);
  if (tokens == 0 && !sums && dS0 == nullptr) return ok();
  seed::ConvArgs a = conv_args(n_seq, channels, width, tokens, cu_seqlens, x, x_stride, io_dtype, weight,
                               bias, S0, activation);
  a.dy = {dy, dy_stride};
  a.dS = dS;
  a.dx = {dx, dx_stride};
  a.dweight = dweight;
  a.dbias = dbias;
  a.dS0 = dS0;
  a.ws = static_cast<float*>(workspace);
  a.vectors = channels % 8 == 0 && vector_rows(x, x_stride, e) && vector_rows(dy, dy_stride, e) &&
              vector_rows(dx, dx_stride, e);
  return device_status(fn, seed::launch_short_conv_backward(a, static_cast<hipStream_t>(stream)));
}

size_t seed_short_conv_workspace_bytes(int n_seq, int channels, int width, int tokens) {
  if (check_conv("seed_short_conv_workspace_bytes", n_seq, channels, width, tokens, &n_seq, SEED_F32,
                 SEED_ACT_NONE) != SEED_OK)
    return static_cast<size_t>(-1);
  ok();
  return (size_t)seed::short_conv_parts(n_seq, channels, tokens) * (width + 1) * channels * 4;
}

seed_status seed_short_conv_step(int batch, int channels, int width, const void* x,
                                 long long x_stride, int io_dtype, const float* weight,
                                 const float* bias, const void* S0, int activation, void* y,
                                 long long y_stride, void* S, void* stream) {
  const char* fn = "seed_short_conv_step";
  if (batch < 0) return fail(SEED_E_SHAPE, "%s: batch must be at least 0 (got %d)", fn, batch);
  // (a block or more for each sequence)
  SEED_TRY(check_conv(fn, batch == 0 ? 1 : batch, channels, width, batch, nullptr, io_dtype, activation));
  if (batch == 0) return ok();
  const size_t e = io_dtype == SEED_BF16 ? 2 : 4, T = (size_t)batch, C = (size_t)channels;
  const size_t state = T * (width - 1) * C;
  const Array out[] = {{"y", y, T, C, e, y_stride, true, e}, dense("S", S, state, e, true)};
  const Array rows[] = {{"x", x, T, C, e, x_stride, true, e}, dense("S0", S0, state, e, true)};
  // y may take the place of x, and S that of S0
  for (int i = 0; i < 2; ++i) {
    SEED_TRY(check_array(fn, rows[i]));
    const bool y_there = i == 0 && y == x && y_stride == x_stride, S_there = i == 1 && S == S0;
    if (!y_there && overlap(out[0], rows[i])) return fail(SEED_E_ARG, "%s: y overlaps %s", fn, rows[i].name);
    if (!S_there && overlap(out[1], rows[i])) return fail(SEED_E_ARG, "%s: S overlaps %s", fn, rows[i].name);
  }
  const Array in[] = {dense("weight", weight, C * width, 4, true), dense("bias", bias, C, 4, false)};
  SEED_TRY(check_arrays(fn, out, in));
  seed::ConvArgs a = conv_args(batch, channels, width, batch, nullptr, x, x_stride, io_dtype, weight, bias,
                               S0, activation);
  a.y = {y, y_stride};
  a.S = S;
  a.vectors = channels % 8 == 0 && vector_rows(x, x_stride, e) && vector_rows(y, y_stride, e);
  return device_status(fn, seed::launch_short_conv_step(a, static_cast<hipStream_t>(stream)));
}

seed_status seed_selective_scan(int n_seq, int channels, int groups, int d_state, int tokens,
                                const int* cu_seqlens, const void* x, long long x_stride,
                                const void* dt, long long dt_stride, const float* A, const void* B,
                                long long B_stride, const void* C, long long C_stride,
                                int io_dtype, const float* D, const void* z, long long z_stride,
                                const float* dt_bias, int softplus, const float* S0, void* y,
                                long long y_stride, float* S, void* workspace,
                                size_t workspace_bytes, void* stream) {
  const char* fn = "seed_selective_scan";
  SEED_TRY(check_select(fn, n_seq, channels, groups, d_state, tokens, cu_seqlens, io_dtype));
  const size_t e = io_dtype == SEED_BF16 ? 2 : 4, T = (size_t)tokens, W = (size_t)channels;
  const size_t bc = (size_t)groups * d_state, state = (size_t)n_seq * W * d_state;
  const size_t want = seed_selective_scan_workspace_bytes(n_seq, channels, groups, d_state, tokens, 0);
  const Array out[] = {{"y", y, T, W, e, y_stride, true, e}, dense("S", S, state, 4, true),
                       dense("workspace", workspace, want, 1, want > 0)};
  Array in[] = {{"x", x, T, W, e, x_stride, true, e},
                {"dt", dt, T, W, e, dt_stride, true, e},
                {"B", B, T, bc, e, B_stride, true, e},
                {"C", C, T, bc, e, C_stride, true, e},
                {"z", z, T, W, e, z_stride, false, e},
                dense("A", A, W * d_state, 4, true),
                dense("D", D, W, 4, false),
                dense("dt_bias", dt_bias, W, 4, false),
                dense("S0", S0, state, 4, false),
                dense("cu_seqlens", cu_seqlens, (size_t)n_seq + 1, 4, false)};
  in[9].align = 4;
  if (S0 != nullptr && S == S0) {
    SEED_TRY(check_array(fn, in[8]));
    in[8].p = nullptr;
  }
  SEED_TRY(check_arrays(fn, out, in));
  if (workspace_bytes < want)
    return fail(SEED_E_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, want);
  seed::SelectArgs a = select_args(n_seq, channels, groups, d_state, tokens, cu_seqlens, x, x_stride, dt,
                                   dt_stride, A, B, B_stride, C, C_stride, io_dtype, D, z, z_stride,
                                   dt_bias, softplus, S0);
  a.y = {y, y_stride};
  a.S = S;
  a.ws = static_cast<char*>(workspace);
  a.at = seed::select_layout(n_seq, channels, groups, d_state, tokens, false);
  return device_status(fn, seed::launch_select(a, static_cast<hipStream_t>(stream)));
}

seed_status seed_selective_scan_backward(
    int n_seq, int channels, int groups, int d_state, int tokens, const int* cu_seqlens,
    const void* x, long long x_stride, const void* dt, long long dt_stride, const float* A,
    const void* B, long long B_stride, const void* C, long long C_stride, int io_dtype,
    const float* D, const void* z, long long z_stride, const float* dt_bias, int softplus,
    const float* S0, const void* dy, long long dy_stride, const float* dS, void* dx,
    long long dx_stride, void* ddt, long long ddt_stride, float* dA, void* dB, long long dB_stride,
    void* dC, long long dC_stride, float* dD, void* dz, long long dz_stride, float* ddt_bias,
    float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "seed_selective_scan_backward";
  SEED_TRY(check_select(fn, n_seq, channels, groups, d_state, tokens, cu_seqlens, io_dtype));
  if (tokens > 0 && (z != nullptr) != (dz != nullptr))
    return fail(SEED_E_ARG, "%s: dz must be given exactly if z is", fn);
  const size_t e = io_dtype == SEED_BF16 ? 2 : 4, T = (size_t)tokens, W = (size_t)channels;
  const size_t bc = (size_t)groups * d_state, state = (size_t)n_seq * W * d_state;
  const size_t want = seed_selective_scan_workspace_bytes(n_seq, channels, groups, d_state, tokens, 1);
  const Array out[] = {{"dx", dx, T, W, e, dx_stride, true, e},
                       {"ddt", ddt, T, W, e, ddt_stride, true, e},
                       {"dB", dB, T, bc, e, dB_stride, true, e},
                       {"dC", dC, T, bc, e, dC_stride, true, e},
                       {"dz", dz, T, W, e, dz_stride, false, e},
                       dense("dA", dA, W * d_state, 4, true),
                       dense("dD", dD, W, 4, false),
                       dense("ddt_bias", ddt_bias, W, 4, false),
                       dense("dS0", dS0, state, 4, false),
                       dense("workspace", workspace, want, 1, want > 0)};
  Array in[] = {{"x", x, T, W, e, x_stride, true, e},
                {"dt", dt, T, W, e, dt_stride, true, e},
                {"B", B, T, bc, e, B_stride, true, e},
                {"C", C, T, bc, e, C_stride, true, e},
                {"z", z, T, W, e, z_stride, false, e},
                {"dy", dy, T, W, e, dy_stride, true, e},
                dense("A", A, W * d_state, 4, true),
                dense("D", D, W, 4, false),
                dense("dt_bias", dt_bias, W, 4, false),
                dense("S0", S0, state, 4, false),
                dense("dS", dS, state, 4, false),
                dense("cu_seqlens", cu_seqlens, (size_t)n_seq + 1, 4, false)};
  in[11].align = 4;
  if (dS0 != nullptr && dS0 == dS) {
    SEED_TRY(check_array(fn, in[10]));
    in[10].p = nullptr;
  }
  SEED_TRY(check_arrays(fn, out, in));
  if (workspace_bytes < want)
    return fail(SEED_E_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, want);
  seed::SelectArgs a = select_args(n_seq, channels, groups, d_state, tokens, cu_seqlens, x, x_stride, dt,
                                   dt_stride, A, B, B_stride, C, C_stride, io_dtype, D, z, z_stride,
                                   dt_bias, softplus, S0);
  a.dy = {dy, dy_stride};
  a.dS = dS;
  a.dx = {dx, dx_stride};
  a.ddt = {ddt, ddt_stride};
  a.dB = {dB, dB_stride};
  a.dC = {dC, dC_stride};
  a.dz = {dz, dz_stride};
  a.dA = dA;
  a.dD = dD;
  a.ddt_bias = ddt_bias;
  a.dS0 = dS0;
  a.ws = static_cast<char*>(workspace);
  a.at = seed::select_layout(n_seq, channels, groups, d_state, tokens, true);
  return device_status(fn, seed::launch_select_backward(a, static_cast<hipStream_t>(stream)));
}

size_t seed_selective_scan_workspace_bytes(int n_seq, int channels, int groups, int d_state,
                                           int tokens, int backward) {
  if (check_select("seed_selective_scan_workspace_bytes", n_seq, channels, groups, d_state, tokens, &n_seq,
                   SEED_F32) != SEED_OK)
    return static_cast<size_t>(-1);
  ok();
  if (tokens == 0) return 0;
  return seed::select_layout(n_seq, channels, groups, d_state, tokens, backward != 0).bytes;
}

seed_status seed_selective_step(int batch, int channels, int groups, int d_state, const void* x,
                                long long x_stride, const void* dt, long long dt_stride,
                                const float* A, const void* B, long long B_stride, const void* C,
                                long long C_stride, int io_dtype, const float* D, const void* z,
                                long long z_stride, const float* dt_bias, int softplus,
                                const float* S0, void* y, long long y_stride, float* S,
                                void* stream) {
  const char* fn = "seed_selective_step";
  if (batch < 0) return fail(SEED_E_SHAPE, "%s: batch must be at least 0 (got %d)", fn, batch);
  SEED_TRY(check_select(fn, 1, channels, groups, d_state, batch, nullptr, io_dtype));
  if (batch == 0) return ok();
  const size_t e = io_dtype == SEED_BF16 ? 2 : 4, T = (size_t)batch, W = (size_t)channels;
  const size_t bc = (size_t)groups * d_state, state = T * W * d_state;
  const Array out[] = {{"y", y, T, W, e, y_stride, true, e}, dense("S", S, state, 4, true)};
  const Array rows[] = {{"x", x, T, W, e, x_stride, true, e},
                        {"dt", dt, T, W, e, dt_stride, true, e},
                        {"z", z, T, W, e, z_stride, false, e},
                        dense("S0", S0, state, 4, true)};
  // y may take the place of x, dt or z, and S that of S0
  for (int i = 0; i < 4; ++i) {
    SEED_TRY(check_array(fn, rows[i]));
    const bool y_there = i < 3 && y == rows[i].p && y_stride == rows[i].stride;
    const bool S_there = i == 3 && S == S0;
    if (!y_there && overlap(out[0], rows[i])) return fail(SEED_E_ARG, "%s: y overlaps %s", fn, rows[i].name);
    if (!S_there && overlap(out[1], rows[i])) return fail(SEED_E_ARG, "%s: S overlaps %s", fn, rows[i].name);
  }
  const Array in[] = {{"B", B, T, bc, e, B_stride, true, e},
                      {"C", C, T, bc, e, C_stride, true, e},
                      dense("A", A, W * d_state, 4, true),
                      dense("D", D, W, 4, false),
                      dense("dt_bias", dt_bias, W, 4, false)};
  SEED_TRY(check_arrays(fn, out, in));
  seed::SelectArgs a = select_args(batch, channels, groups, d_state, batch, nullptr, x, x_stride, dt, dt_stride,
                                   A, B, B_stride, C, C_stride, io_dtype, D, z, z_stride, dt_bias, softplus,
                                   S0);
  a.y = {y, y_stride};
  a.S = S;
  return device_status(fn, seed::launch_select_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
