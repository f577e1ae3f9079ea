// The recurrence over sequences: workspace layout and the order of its phases.
#include "seed_scan.h"

namespace seed {

ScanLayout scan_layout(int rule, int n_seq, int heads, int key_heads, int d_k, int d_v, int tokens,
                       bool backward) {
  const bool kda = rule == kKDA, delta = rule != kMAMBA2;
  const size_t slots = (size_t)(tokens / kScanChunk) + (size_t)n_seq;
  const size_t units = slots * heads;
  size_t at = 0;
  auto part = [&](bool used, size_t bytes) {
    const size_t here = at;
    if (used) at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t pack = (size_t)6 * 3 * 512 * 2;
  const size_t per_token = units * kScanChunk * sizeof(float);
  const size_t per_head = (size_t)tokens * heads * d_k * sizeof(float);
  ScanLayout l{};
  l.n_pack = part(delta, units * pack);
  l.nt_pack = part(delta && backward, units * pack);
  l.m_pack = part(true, units * pack);
  l.vec = part(true, 4 * per_token);
  l.p = part(kda, per_token * d_k);
  l.f = part(kda, per_token * d_k);
  l.state = part(backward, units * d_k * d_v * sizeof(float));
  l.grad = part(backward, units * d_k * d_v * sizeof(float));
  l.e = part(backward && delta, per_token * d_v);
  l.y = part(backward && delta, per_token * d_v);
  l.dq = part(backward && (kda || heads != key_heads), per_head);
  l.dk = part(backward && (kda || heads != key_heads), per_head);
  l.tp = part(backward && kda, per_token * d_k);
  l.tf = part(backward && kda, per_token * d_k);
  l.slow = part(backward && kda, units * sizeof(int));
  // Few units and a long axis: segments of it run side by side, each from a
  // start that a first pass over the others' carries gives.  The first pass
  // and the second each cost what the whole would, so segments pay where
  // whole sequences fill at most a quarter of the CUs (a workgroup has 64
  // columns): 16 heads of 64 x 64 over 256 chunks took 1655 us whole and take
  // 240 in segments; 128 workgroups of 32 chunks were slower in segments.
  const long long groups = (long long)n_seq * heads * (d_v / 64);
  const int chunks = tokens / kScanChunk / (n_seq > 0 ? n_seq : 1);
  if (groups <= 64 && chunks >= 8) {
    const int wanted = (int)(256 / groups), each = (chunks + wanted - 1) / wanted;
    l.seg = each < 4 ? 4 : each;
    l.segs = tokens / (kScanChunk * l.seg) + n_seq;
  }
  const size_t seg_units = (size_t)l.segs * heads;
  l.carry = part(l.seg > 0, seg_units * d_k * d_v * sizeof(float));
  l.trans = part(l.seg > 0, seg_units * (delta ? d_k * d_k : 1) * sizeof(float));
  l.start = part(l.seg > 0, seg_units * d_k * d_v * sizeof(float));
  l.bytes = at;
  return l;
}

static hipError_t one_walk(const ScanArgs& a, int what, hipStream_t stream) {
  return a.bf16 && a.rule != kKDA ? launch_scan_chain(a, what, stream)
                                  : launch_scan_wide(a, what, stream);
}

static hipError_t walk(const ScanArgs& a, int what, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.at.seg > 0 && a.tokens > 0) {
    // backward, the carries are the forward pass's
    e = one_walk(a, what == 2 ? 4 : 3, stream);
    if (e == hipSuccess) e = launch_scan_join(a, what == 2, stream);
  }
  return e == hipSuccess ? one_walk(a, what, stream) : e;
}

hipError_t launch_scan(const ScanArgs& a, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.tokens > 0) e = launch_scan_prep(a, false, stream);
  if (e == hipSuccess) e = walk(a, 0, stream);
  return e;
}

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.tokens > 0) e = launch_scan_prep(a, true, stream);
  if (e == hipSuccess && a.tokens > 0) e = walk(a, 1, stream);
  if (e == hipSuccess) e = walk(a, 2, stream);
  if (e == hipSuccess && a.tokens > 0) e = launch_scan_grads(a, stream);
  return e;
}

}  // namespace seed
