// C ABI of the operators over sequences (declared in
// include/seed_sequence.h): host validation, then the launchers.
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/seed_sequence.h"
#include "seed_error.h"
#include "seed_sequence_launch.h"

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

seed_status need(const char* fn, const char* name, const void* p) {
  if (p == nullptr) return fail(SEED_E_ARG, "%s: %s is NULL", fn, name);
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0)
    return fail(SEED_E_ARG, "%s: %s is not 16-byte aligned", fn, name);
  return SEED_OK;
}
seed_status need_if(const char* fn, const char* name, const void* p) {
  return p == nullptr ? SEED_OK : need(fn, name, p);
}

#define SEED_TRY(call)              \
  do {                              \
    const seed_status s_ = (call);  \
    if (s_ != SEED_OK) return s_;   \
  } while (0)
#define SEED_NEED(p) SEED_TRY(need(fn, #p, p))
#define SEED_MAY(p) SEED_TRY(need_if(fn, #p, p))

bool known_rule(int rule) {
  return rule == SEED_RULE_GDN || rule == SEED_RULE_KDA || rule == SEED_RULE_MAMBA2;
}
bool known_dtype(int t) { return t == SEED_F32 || t == SEED_BF16; }

// Bytes [p, p + n) against [q, q + m); NULL overlaps nothing.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p != nullptr && q != nullptr && n > 0 && m > 0 && a < b + m && b < a + n;
}

struct Part {
  const char* name;
  const void* p;
  size_t n;
};

seed_status check_shape(const char* fn, int rule, int n_seq, int heads, int key_heads, int d_k,
                        int d_v, int tokens) {
  if (!known_rule(rule)) return fail(SEED_E_ARG, "%s: unknown rule %d", fn, rule);
  if (n_seq <= 0 || heads <= 0 || key_heads <= 0 || d_k <= 0 || d_v <= 0 || tokens < 0)
    return fail(SEED_E_SHAPE,
                "%s: n_seq, heads, key_heads, d_k, d_v must be positive and tokens at least 0 (got "
                "%d, %d, %d, %d, %d, %d)",
                fn, n_seq, heads, key_heads, d_k, d_v, tokens);
  if (heads % key_heads != 0)
    return fail(SEED_E_SHAPE, "%s: heads (%d) must be a multiple of key_heads (%d)", fn, heads,
                key_heads);
  if (!((d_k == 128 && d_v == 128) || (d_k == 128 && d_v == 64) || (d_k == 64 && d_v == 64)))
    return fail(SEED_E_UNSUPPORTED,
                "%s: head shape d_k=%d d_v=%d not supported (use 128x128, 128x64 or 64x64)", fn,
                d_k, d_v);
  if (heads > 65535)
    return fail(SEED_E_UNSUPPORTED, "%s: %d heads exceed the grid limit of 65535", fn, heads);
  // at most 1024 threads for each (chunk or sequence, head), 2^32 in a grid
  const long long slots = (long long)tokens / seed::kScanChunk + n_seq;
  if ((long long)tokens + 64LL * n_seq > 0x7fffffffLL ||
      slots > 0xffffffffLL / 1024 / heads)
    return fail(SEED_E_UNSUPPORTED, "%s: n_seq * heads or tokens * heads exceed the grid limit", fn);
  return SEED_OK;
}

seed_status check_scan(const char* fn, int rule, int n_seq, int heads, int key_heads, int d_k,
                       int d_v, int tokens, const int* cu_seqlens, const void* q, const void* k,
                       const void* v, int in_dtype, const float* g, const float* beta,
                       const float* S0, void* workspace, size_t workspace_bytes, bool backward) {
  SEED_TRY(check_shape(fn, rule, n_seq, heads, key_heads, d_k, d_v, tokens));
  if (!known_dtype(in_dtype)) return fail(SEED_E_ARG, "%s: unknown input dtype %d", fn, in_dtype);
  if (cu_seqlens == nullptr && tokens % n_seq != 0)
    return fail(SEED_E_SHAPE, "%s: %d tokens do not make %d equal sequences", fn, tokens, n_seq);
  SEED_MAY(S0);
  if (cu_seqlens != nullptr && (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0)
    return fail(SEED_E_ARG, "%s: cu_seqlens is not 4-byte aligned", fn);
  if (rule == SEED_RULE_MAMBA2 && beta != nullptr)
    return fail(SEED_E_ARG, "%s: beta must be NULL for Mamba-2", fn);
  if (tokens > 0) {
    SEED_NEED(q);
    SEED_NEED(k);
    SEED_NEED(v);
    SEED_NEED(g);
    if (rule != SEED_RULE_MAMBA2) SEED_NEED(beta);
    const size_t want = seed::scan_layout(rule, n_seq, heads, key_heads, d_k, d_v, tokens, backward).bytes;
    SEED_NEED(workspace);
    if (workspace_bytes < want)
      return fail(SEED_E_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, want);
  }
  return SEED_OK;
}

seed::ScanArgs scan_args(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v,
                         int tokens, const int* cu_seqlens, const void* q, const void* k,
                         const void* v, int in_dtype, const float* g, const float* beta,
                         const float* S0, void* workspace, bool backward) {
  seed::ScanArgs a{};
  a.rule = rule;
  a.bf16 = in_dtype == SEED_BF16;
  a.n_seq = n_seq;
  a.heads = heads;
  a.key_heads = key_heads;
  a.d_k = d_k;
  a.d_v = d_v;
  a.tokens = tokens;
  a.cu = cu_seqlens;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.S0 = S0;
  a.ws = static_cast<char*>(workspace);
  a.at = seed::scan_layout(rule, n_seq, heads, key_heads, d_k, d_v, tokens, backward);
  a.slots = tokens / seed::kScanChunk + n_seq;
  return a;
}

// Outputs against everything else: `out` must not touch `in`, nor each
// other.
seed_status check_overlap(const char* fn, const Part* out, int n_out, const Part* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i].p, out[i].n, in[j].p, in[j].n))
        return fail(SEED_E_ARG, "%s: %s overlaps %s", fn, out[i].name, in[j].name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(SEED_E_ARG, "%s: %s overlaps %s", fn, out[i].name, out[j].name);
  }
  return SEED_OK;
}

seed_status check_norm(const char* fn, long long rows, int groups, int d, int x_dtype,
                       const void* gate, int io_dtype, const float* weight, const float* bias,
                       int weight_groups, float eps, int activation, int gate_first) {
  if (rows < 0 || groups <= 0 || d <= 0)
    return fail(SEED_E_SHAPE, "%s: groups and d must be positive, rows at least 0 (got %lld, %d, %d)",
                fn, rows, groups, d);
  if (weight_groups != 1 && weight_groups != groups)
    return fail(SEED_E_SHAPE, "%s: weight_groups must be 1 or groups = %d (got %d)", fn, groups,
                weight_groups);
  if (d > 8192) return fail(SEED_E_UNSUPPORTED, "%s: %d channels a group, above 8192", fn, d);
  if (groups > 65535)
    return fail(SEED_E_UNSUPPORTED, "%s: %d groups exceed the grid limit of 65535", fn, groups);
  if (rows > 0x7fffffffLL || rows * groups > 0x7fffffffLL)
    return fail(SEED_E_UNSUPPORTED, "%s: rows * groups exceeds the grid limit", fn);
  if (!known_dtype(x_dtype) || !known_dtype(io_dtype))
    return fail(SEED_E_ARG, "%s: unknown dtype (x %d, io %d)", fn, x_dtype, io_dtype);
  if (activation != SEED_ACT_NONE && activation != SEED_ACT_SILU && activation != SEED_ACT_SIGMOID)
    return fail(SEED_E_ARG, "%s: unknown activation %d", fn, activation);
  if (gate_first && gate == nullptr) return fail(SEED_E_ARG, "%s: gate_first without a gate", fn);
  if (!(eps >= 0.f)) return fail(SEED_E_ARG, "%s: eps must be at least 0 (got %g)", fn, (double)eps);
  SEED_MAY(gate);
  SEED_MAY(weight);
  SEED_MAY(bias);
  return SEED_OK;
}

// Columns of a partial sum of dweight and dbias.
size_t norm_columns(int weight_groups, int d) { return ((size_t)weight_groups * 2 * d + 3) & ~(size_t)3; }

seed::NormArgs norm_args(long long rows, int groups, int d, const void* x, int x_dtype,
                         const void* gate, int io_dtype, const float* weight, const float* bias,
                         int weight_groups, float eps, int centered, int activation,
                         int gate_first) {
  seed::NormArgs a{};
  a.rows = rows;
  a.groups = groups;
  a.d = d;
  a.x_bf16 = x_dtype == SEED_BF16;
  a.io_bf16 = io_dtype == SEED_BF16;
  a.x = x;
  a.gate = gate;
  a.weight = weight;
  a.bias = bias;
  a.weight_groups = weight_groups;
  a.eps = eps;
  a.centered = centered != 0;
  a.gate_first = gate_first != 0;
  a.act = activation;
  return a;
}

}  // namespace

extern "C" {

seed_status seed_scan(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v, int tokens,
                      const int* cu_seqlens, const void* q, const void* k, const void* v,
                      int in_dtype, const float* g, const float* beta, const float* S0, void* o,
                      float* S, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "seed_scan";
  SEED_TRY(check_scan(fn, rule, n_seq, heads, key_heads, d_k, d_v, tokens, cu_seqlens, q, k, v,
                      in_dtype, g, beta, S0, workspace, workspace_bytes, false));
  SEED_NEED(S);
  if (tokens > 0) SEED_NEED(o);
  const size_t e = in_dtype == SEED_BF16 ? 2 : 4, T = (size_t)tokens;
  const size_t state = (size_t)n_seq * heads * d_k * d_v * 4;
  const Part out[] = {{"o", o, T * heads * d_v * e}, {"S", S, state}, {"workspace", workspace, workspace_bytes}};
  const Part in[] = {{"q", q, T * key_heads * d_k * e},
                     {"k", k, T * key_heads * d_k * e},
                     {"v", v, T * heads * d_v * e},
                     {"g", g, T * heads * (rule == SEED_RULE_KDA ? d_k : 1) * 4},
                     {"beta", beta, T * heads * 4},
                     {"S0", S == S0 ? nullptr : S0, state},
                     {"cu_seqlens", cu_seqlens, ((size_t)n_seq + 1) * sizeof(int)}};
  SEED_TRY(check_overlap(fn, out, 3, in, 7));
  seed::ScanArgs a = scan_args(rule, n_seq, heads, key_heads, d_k, d_v, tokens, cu_seqlens, q, k, v,
                               in_dtype, g, beta, S0, workspace, false);
  a.o = o;
  a.S = S;
  return device_status(fn, seed::launch_scan(a, static_cast<hipStream_t>(stream)));
}

seed_status seed_scan_backward(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v,
                               int tokens, const int* cu_seqlens, const void* q, const void* k,
                               const void* v, int in_dtype, const float* g, const float* beta,
                               const float* S0, const void* dO, const float* dS, void* dq,
                               void* dk, void* dv, float* dg, float* dbeta, float* dS0,
                               void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "seed_scan_backward";
  SEED_TRY(check_scan(fn, rule, n_seq, heads, key_heads, d_k, d_v, tokens, cu_seqlens, q, k, v,
                      in_dtype, g, beta, S0, workspace, workspace_bytes, true));
  SEED_MAY(dS);
  SEED_MAY(dS0);
  if (rule == SEED_RULE_MAMBA2 && dbeta != nullptr)
    return fail(SEED_E_ARG, "%s: dbeta must be NULL for Mamba-2", fn);
  if (tokens > 0) {
    SEED_NEED(dO);
    SEED_NEED(dq);
    SEED_NEED(dk);
    SEED_NEED(dv);
    SEED_NEED(dg);
    if (rule != SEED_RULE_MAMBA2) SEED_NEED(dbeta);
  }
  const size_t e = in_dtype == SEED_BF16 ? 2 : 4, T = (size_t)tokens;
  const size_t state = (size_t)n_seq * heads * d_k * d_v * 4, keys = T * key_heads * d_k * e;
  const size_t values = T * heads * d_v * e, gates = T * heads * (rule == SEED_RULE_KDA ? d_k : 1) * 4;
  const Part out[] = {{"dq", dq, keys}, {"dk", dk, keys}, {"dv", dv, values}, {"dg", dg, gates},
                      {"dbeta", dbeta, T * heads * 4}, {"dS0", dS0, state},
                      {"workspace", workspace, workspace_bytes}};
  const Part in[] = {{"q", q, keys}, {"k", k, keys}, {"v", v, values}, {"g", g, gates},
                     {"beta", beta, T * heads * 4}, {"S0", S0, state}, {"dO", dO, values},
                     {"dS", dS0 == dS ? nullptr : dS, state},
                     {"cu_seqlens", cu_seqlens, ((size_t)n_seq + 1) * sizeof(int)}};
  SEED_TRY(check_overlap(fn, out, 7, in, 9));
  seed::ScanArgs a = scan_args(rule, n_seq, heads, key_heads, d_k, d_v, tokens, cu_seqlens, q, k, v,
                               in_dtype, g, beta, S0, workspace, true);
  a.dO = dO;
  a.dS = dS;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dS0 = dS0;
  return device_status(fn, seed::launch_scan_backward(a, static_cast<hipStream_t>(stream)));
}

size_t seed_scan_workspace_bytes(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v,
                                 int tokens, int backward) {
  if (check_shape("seed_scan_workspace_bytes", rule, n_seq, heads, key_heads, d_k, d_v, tokens) !=
      SEED_OK)
    return static_cast<size_t>(-1);
  ok();
  if (tokens == 0) return 0;
  return seed::scan_layout(rule, n_seq, heads, key_heads, d_k, d_v, tokens, backward != 0).bytes;
}

seed_status seed_group_norm(long long rows, int groups, int d, const void* x, int x_dtype,
                            const void* gate, int io_dtype, const float* weight,
                            const float* bias, int weight_groups, float eps, int centered,
                            int activation, int gate_first, void* y, void* stream) {
  const char* fn = "seed_group_norm";
  SEED_TRY(check_norm(fn, rows, groups, d, x_dtype, gate, io_dtype, weight, bias, weight_groups,
                      eps, activation, gate_first));
  if (rows == 0) return ok();
  SEED_NEED(x);
  SEED_NEED(y);
  const size_t N = (size_t)rows * groups * d;
  const size_t xb = N * (x_dtype == SEED_BF16 ? 2 : 4), io = N * (io_dtype == SEED_BF16 ? 2 : 4);
  const size_t wb = (size_t)weight_groups * d * 4;
  const Part out[] = {{"y", y, io}};
  const Part in[] = {{"x", y == x && x_dtype == io_dtype ? nullptr : x, xb},
                     {"gate", y == gate ? nullptr : gate, io},
                     {"weight", weight, wb},
                     {"bias", bias, wb}};
  SEED_TRY(check_overlap(fn, out, 1, in, 4));
  seed::NormArgs a = norm_args(rows, groups, d, x, x_dtype, gate, io_dtype, weight, bias,
                               weight_groups, eps, centered, activation, gate_first);
  a.y = y;
  return device_status(fn, seed::launch_group_norm(a, static_cast<hipStream_t>(stream)));
}

seed_status seed_group_norm_backward(long long rows, int groups, int d, const void* dy,
                                     const void* x, int x_dtype, const void* gate, int io_dtype,
                                     const float* weight, const float* bias, int weight_groups,
                                     float eps, int centered, int activation, int gate_first,
                                     void* dx, void* dgate, float* dweight, float* dbias,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "seed_group_norm_backward";
  SEED_TRY(check_norm(fn, rows, groups, d, x_dtype, gate, io_dtype, weight, bias, weight_groups,
                      eps, activation, gate_first));
  if ((gate != nullptr) != (dgate != nullptr) && rows > 0)
    return fail(SEED_E_ARG, "%s: dgate must be given exactly if gate is", fn);
  SEED_MAY(dgate);
  SEED_MAY(dweight);
  SEED_MAY(dbias);
  if (rows > 0) {
    SEED_NEED(dy);
    SEED_NEED(x);
    SEED_NEED(dx);
  }
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (rows == 0 && !sums) return ok();
  const int parts = seed::group_norm_parts(rows, groups, d, weight_groups);
  const size_t want = sums ? (size_t)parts * norm_columns(weight_groups, d) * 4 : 0;
  if (sums) {
    SEED_NEED(workspace);
    if (workspace_bytes < want)
      return fail(SEED_E_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, want);
  }
  const size_t N = (size_t)rows * groups * d;
  const size_t xb = N * (x_dtype == SEED_BF16 ? 2 : 4), io = N * (io_dtype == SEED_BF16 ? 2 : 4);
  const size_t wb = (size_t)weight_groups * d * 4;
  const bool same = x_dtype == io_dtype;
  const Part out[] = {{"dx", dx, xb}, {"dgate", dgate, io}, {"dweight", dweight, wb},
                      {"dbias", dbias, wb}, {"workspace", sums ? workspace : nullptr, want}};
  // an output may take the place of an input element for element
  for (const Part& o : out) {
    const Part in[] = {
        {"x", o.p == dx && dx == x ? nullptr : x, xb},
        {"dy", (o.p == dx && dx == dy && same) || (o.p == dgate && dgate == dy) ? nullptr : dy, io},
        {"gate", o.p == dgate && dgate == gate ? nullptr : gate, io},
        {"weight", weight, wb},
        {"bias", bias, wb}};
    SEED_TRY(check_overlap(fn, &o, 1, in, 5));
  }
  SEED_TRY(check_overlap(fn, out, 5, nullptr, 0));
  seed::NormArgs a = norm_args(rows, groups, d, x, x_dtype, gate, io_dtype, weight, bias,
                               weight_groups, eps, centered, activation, gate_first);
  a.dy = dy;
  a.dx = dx;
  a.dgate = dgate;
  a.dweight = dweight;
  a.dbias = dbias;
  a.ws = static_cast<float*>(workspace);
  a.parts = parts;
  return device_status(fn, seed::launch_group_norm_backward(a, static_cast<hipStream_t>(stream)));
}

size_t seed_group_norm_workspace_bytes(long long rows, int groups, int d, int weight_groups) {
  if (check_norm("seed_group_norm_workspace_bytes", rows, groups, d, SEED_F32, nullptr, SEED_F32,
                 nullptr, nullptr, weight_groups, 0.f, SEED_ACT_NONE, 0) != SEED_OK)
    return static_cast<size_t>(-1);
  ok();
  return (size_t)seed::group_norm_parts(rows, groups, d, weight_groups) * norm_columns(weight_groups, d) * 4;
}

}  // extern "C"
