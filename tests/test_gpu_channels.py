"""The operators on channels together, and with the heads' operators, as
layers use them.

A selective layer: projection rows -> short convolution -> selective scan with
its gate, for prompts and single tokens, and in training.  A Gated DeltaNet
layer: projection rows -> convolutions of q, k and v -> the recurrence over
sequences -> decode steps from its states.  Each operator is checked against
the float64 oracle from the very values it was given, so its own bounds hold
(oracle/seed_channels.py, test_gpu_scan.py)."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_channels as och
from oracle import seed_sequence as oseq
from sink_rank_recurrent_amd import binding, channels, sequence
from test_gpu_scan import check as check_scan
from test_gpu_selective_scan import depth as scan_depth
from test_gpu_short_conv import check, depth, half

pytestmark = [pytest.mark.gpu, requires_gpu]

W, N, G, K = 96, 16, 2, 4


def weights(seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    return normal, {"conv": normal(W, K) / 2, "bias": 0.2 * normal(W), "A": -torch.exp(0.5 * normal(W, N)),
                    "D": normal(W), "dt_bias": 0.5 * normal(W) - 1}


def layer(p, xz, dt, bc, cu, held, S):
    """Prompts through the layer, its states in place; what lies between and
    the result."""
    T = xz.shape[0]
    n = cu.shape[0] - 1
    u, y = torch.empty(T, W, device="cuda", dtype=xz.dtype), torch.empty(T, W, device="cuda", dtype=xz.dtype)
    channels.seed_short_conv(xz[:, :W], p["conv"], u, bias=p["bias"], S0=held, S=held, cu_seqlens=cu)
    channels.seed_selective_scan(u, dt, p["A"], bc[:, 0], bc[:, 1], y, S, D=p["D"], z=xz[:, W:],
                                 dt_bias=p["dt_bias"], S0=S, cu_seqlens=cu)
    return u, y


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_selective_layer_serving(dtype):
    """Prompts of 1, 0, 7 and 300 tokens, then five decode steps of all
    requests, each operator from the values that it was given."""
    offsets = [0, 1, 1, 8, 308]
    B, T = 4, 308
    normal, p = weights(1)
    io = 0.0 if dtype == torch.float32 else half(dtype)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    held, S = torch.zeros(B, K - 1, W, device="cuda", dtype=dtype), torch.zeros(B, W, N, device="cuda")
    h = {k: f64(v) for k, v in p.items()}

    def inputs(rows):
        return normal(rows, 2 * W).to(dtype), normal(rows, W).to(dtype), normal(rows, 2, G, N).to(dtype)

    def against(xz, dt, bc, u, y, before, at):
        """The oracle from the states `before`; the states behind are the kernels'."""
        x, z = f64(xz[:, :W]), f64(xz[:, W:])
        want, off, kept = och.conv(x, h["conv"], h["bias"], before[0], True, at, io)
        check(u, want, off, "u")
        assert np.array_equal(f64(held), kept)
        (want, off), (wS, S_off) = och.select(f64(u), f64(dt), h["A"], f64(bc[:, 0]), f64(bc[:, 1]), h["D"], z,
                                              h["dt_bias"], True, before[1], at, io)
        check(y, want, off, "y")
        check(S, wS, S_off, "S")

    xz, dt, bc = inputs(T)
    before = f64(held), f64(S)
    u, y = layer(p, xz, dt, bc, cu, held, S)
    against(xz, dt, bc, u, y, before, offsets)
    for _ in range(5):
        xz, dt, bc = inputs(B)
        before = f64(held), f64(S)
        u, y = torch.empty(B, W, device="cuda", dtype=dtype), torch.empty(B, W, device="cuda", dtype=dtype)
        channels.seed_short_conv_step(xz[:, :W], p["conv"], u, held, bias=p["bias"])
        channels.seed_selective_step(u, dt, p["A"], bc[:, 0], bc[:, 1], y, S, D=p["D"], z=xz[:, W:],
                                     dt_bias=p["dt_bias"])
        against(xz, dt, bc, u, y, before, list(range(B + 1)))


def test_decode_captured_and_replayed():
    """A decode step of the layer in a graph, its states in place: three
    replays are three eager steps."""
    B = 5
    normal, p = weights(2)
    xz, dt, bc = normal(B, 2 * W).bfloat16(), normal(B, W).bfloat16(), normal(B, 2, G, N).bfloat16()
    first = normal(B, K - 1, W).bfloat16(), normal(B, W, N)

    def step(held, S, u, y):
        channels.seed_short_conv_step(xz[:, :W], p["conv"], u, held, bias=p["bias"])
        channels.seed_selective_step(u, dt, p["A"], bc[:, 0], bc[:, 1], y, S, D=p["D"], z=xz[:, W:],
                                     dt_bias=p["dt_bias"])

    def state():
        return [first[0].clone(), first[1].clone(), torch.zeros(B, W, device="cuda", dtype=torch.bfloat16),
                torch.zeros(B, W, device="cuda", dtype=torch.bfloat16)]

    eager, graph = state(), state()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*graph)
    for t, x in zip(graph, state()):
        t.copy_(x)
    for _ in range(3):
        step(*eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, graph))
        xz.copy_(normal(B, 2 * W))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_selective_layer_training(dtype):
    """Forward and back through scan and convolution, dx and dz into one
    projection's gradient: each pass against the oracle from its inputs."""
    offsets, T = [0, 130, 131, 131, 400], 400
    normal, p = weights(3)
    io = 0.0 if dtype == torch.float32 else half(dtype)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    xz, dt, bc = normal(T, 2 * W).to(dtype), normal(T, W).to(dtype), normal(T, 2, G, N).to(dtype)
    dy = normal(T, W).to(dtype)
    u, y = layer(p, xz, dt, bc, cu, torch.zeros(4, K - 1, W, device="cuda", dtype=dtype),
                 torch.zeros(4, W, N, device="cuda"))
    du, ddt, dxz, dbc = torch.empty_like(u), torch.empty_like(dt), torch.empty_like(xz), torch.empty_like(bc)
    d = {k: torch.empty_like(v) for k, v in p.items()}
    channels.seed_selective_scan_backward(dy, u, dt, p["A"], bc[:, 0], bc[:, 1], du, ddt, d["A"], dbc[:, 0],
                                          dbc[:, 1], D=p["D"], z=xz[:, W:], dt_bias=p["dt_bias"], dD=d["D"],
                                          dz=dxz[:, W:], ddt_bias=d["dt_bias"], cu_seqlens=cu)
    channels.seed_short_conv_backward(du, xz[:, :W], p["conv"], dxz[:, :W], dweight=d["conv"], dbias=d["bias"],
                                      bias=p["bias"], cu_seqlens=cu)
    h = {k: f64(v) for k, v in p.items()}
    want = och.select_backward(f64(u), f64(dt), h["A"], f64(bc[:, 0]), f64(bc[:, 1]), h["D"], f64(xz[:, W:]),
                               h["dt_bias"], True, None, offsets, f64(dy), None, max(scan_depth(offsets, W, G, T)), io)
    for name, got in (("x", du), ("dt", ddt), ("A", d["A"]), ("B", dbc[:, 0]), ("C", dbc[:, 1]), ("D", d["D"]),
                      ("z", dxz[:, W:]), ("dt_bias", d["dt_bias"])):
        check(got, *want[name], name)
    want = och.conv_backward(f64(xz[:, :W]), h["conv"], h["bias"], None, True, offsets, f64(du), None,
                             depth(offsets, T), io)
    for name, got in (("x", dxz[:, :W]), ("weight", d["conv"]), ("bias", d["bias"])):
        check(got, *want[name], name)


def test_delta_layer_serving():
    """Convolutions of q, k and v, slices of one projection, in front of the
    recurrence and of its dense decode steps."""
    H, d_k, B = 2, 64, 3
    offsets, T, C = [0, 2, 2, 80], 80, H * d_k
    gen = torch.Generator("cuda").manual_seed(4)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    weight = [normal(C, K) / 2 for _ in range(3)]
    held = [torch.zeros(B, K - 1, C, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    S = torch.zeros(B, H, d_k, d_k, device="cuda")

    def gates(rows):
        return 0.9 + 0.099 * torch.rand(rows, H, device="cuda", generator=gen), torch.rand(rows, H, device="cuda",
                                                                                           generator=gen)

    def unit(x):      # keys and queries of unit length
        return torch.nn.functional.normalize(x.float(), dim=-1).bfloat16()

    qkv = normal(T, 3 * C).bfloat16()
    out = [torch.empty(T, C, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    for i in range(3):
        channels.seed_short_conv(qkv[:, i * C:(i + 1) * C], weight[i], out[i], S0=held[i], S=held[i], cu_seqlens=cu)
        want, off, kept = och.conv(f64(qkv[:, i * C:(i + 1) * C]), f64(weight[i]), None, None, True, offsets,
                                   half(torch.bfloat16))
        check(out[i], want, off, "qkv"[i])
        assert np.array_equal(f64(held[i]), kept)
    q, k, v = (x.view(T, H, d_k) for x in out)
    q, k = unit(q), unit(k)
    g, beta = gates(T)
    o = torch.empty_like(v)
    sequence.seed_scan("gdn", q, k, v, g, beta, o, S, cu_seqlens=cu)
    want_o, want_S = oseq.scan("gdn", f64(q), f64(k), f64(v), f64(g), f64(beta), None, offsets)
    check_scan(o, want_o, offsets, "o")
    check_scan(S, want_S, [0], "S")
    read = torch.empty(B, H, d_k, device="cuda")
    for _ in range(3):
        qkv = normal(B, 3 * C).bfloat16()
        now = [torch.empty(B, C, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
        for i in range(3):
            before = f64(held[i])
            channels.seed_short_conv_step(qkv[:, i * C:(i + 1) * C], weight[i], now[i], held[i])
            want, off, kept = och.conv(f64(qkv[:, i * C:(i + 1) * C]), f64(weight[i]), None, before, True,
                                       list(range(B + 1)), half(torch.bfloat16))
            check(now[i], want, off, "qkv"[i])
            assert np.array_equal(f64(held[i]), kept)
        q, k, v = (x.view(B, H, d_k) for x in now)
        q, k = unit(q), unit(k)
        g, beta = gates(B)
        before = f64(S)
        binding.dense_decode_step("gdn", S, q, k, v, g, beta, read)
        for b in range(B):
            _, want_S = oseq.scan("gdn", *(f64(t[b:b + 1]) for t in (q, k, v, g, beta)), before[b:b + 1], [0, 1])
            assert np.abs(f64(S[b]) - want_S[0]).max() <= 1e-5 * np.abs(want_S[0]).max()


@pytest.mark.parametrize("op", ["conv", "scan"])
def test_two_streams_at_once(op):
    """Two calls on two streams, each with its own workspace: the bits of one
    after the other."""
    normal, p = weights(5)
    T = 2000
    cu = torch.tensor([0, 700, T], dtype=torch.int32, device="cuda")
    x = [normal(T, W).bfloat16() for _ in range(2)]
    dt, bc, dy = normal(T, W).bfloat16(), normal(T, 2, G, N).bfloat16(), normal(T, W).bfloat16()

    def run(i, stream=None):
        e = torch.empty_like
        if op == "conv":
            out = [e(x[i]), e(x[i]), e(p["conv"]), e(p["bias"])]
            channels.seed_short_conv(x[i], p["conv"], out[0], bias=p["bias"], cu_seqlens=cu, stream=stream)
            channels.seed_short_conv_backward(dy, x[i], p["conv"], out[1], dweight=out[2], dbias=out[3],
                                              bias=p["bias"], cu_seqlens=cu, stream=stream)
            return out
        args = x[i], dt, p["A"], bc[:, 0], bc[:, 1]
        out = [e(x[i]), torch.empty(2, W, N, device="cuda"), e(x[i]), e(dt), e(p["A"]), e(bc[:, 0]), e(bc[:, 1])]
        channels.seed_selective_scan(*args, out[0], out[1], cu_seqlens=cu, stream=stream)
        channels.seed_selective_scan_backward(dy, *args, *out[2:], cu_seqlens=cu, stream=stream)
        return out

    ref = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [run(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_offsets_out_of_order():
    """Offsets that fall, repeat or lie outside are no access outside the
    arrays: what is written lies in the outputs' rows, and the calls end."""
    normal, p = weights(6)
    T = 200
    x, dt, bc = normal(T, W).bfloat16(), normal(T, W).bfloat16(), normal(T, 2, G, N).bfloat16()
    for offsets in ([0, 150, 100, 200], [50, 10, 300, -5], [200, 0, 0, 200], [-7, -7, 1 << 30, 3]):
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        guard = torch.full((T + 64, W), 3.0, device="cuda", dtype=torch.bfloat16)
        y = guard[32:32 + T]
        ends = torch.full((5, W, N), 3.0, device="cuda")
        S = ends[1:4]
        channels.seed_short_conv(x, p["conv"], y, cu_seqlens=cu)
        channels.seed_selective_scan(x, dt, p["A"], bc[:, 0], bc[:, 1], y, S, cu_seqlens=cu)
        dw, db = torch.empty_like(p["conv"]), torch.empty_like(p["bias"])
        channels.seed_short_conv_backward(x, x, p["conv"], y, dweight=dw, dbias=db, cu_seqlens=cu)
        out = [torch.empty_like(t) for t in (dt, p["A"], bc[:, 0], bc[:, 1])]
        channels.seed_selective_scan_backward(x, x, dt, p["A"], bc[:, 0], bc[:, 1], y, out[0], out[1], out[2], out[3],
                                              cu_seqlens=cu)
        torch.cuda.synchronize()
        assert (guard[:32] == 3).all() and (guard[32 + T:] == 3).all()
        assert (ends[0] == 3).all() and (ends[4] == 3).all()
