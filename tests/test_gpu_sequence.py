"""The sequence operators together, as a layer uses them: prompts through the
recurrence into shallow states, the read-outs through the gated norm, decode
steps from the states; in training the layer forward and back.

Tolerances: a prompt's read-outs and states are within F32 = 1.3e-5 of a
unit's largest value (test_gpu_scan.py).  A prompt of at most R tokens has a
state of rank R at most, so its conversion loses nothing but rounding: 1e-4 of
the state's norm (gpu_util.TOL_STATE_COMPRESS); factors rounded to fp16 move
each of R rank-one terms by 2^-10 of its size, sqrt(R) 2^-10 of the norm
together.  A read-out with a query of length 1 is off by no more than its
state; each exact step adds 1e-5 (gpu_util.TOL_STATE_STEP)."""
import numpy as np
import pytest
import torch

from gpu_util import TOL_STATE_COMPRESS, TOL_STATE_STEP, f64, requires_gpu
from oracle import seed_sequence as oseq
from sink_rank_recurrent_amd import binding, sequence
from test_gpu_group_norm import close
from test_gpu_scan import F32, RULES, check, host, inputs

pytestmark = [pytest.mark.gpu, requires_gpu]

R, W, H = 16, 16, 3


@pytest.fixture(autouse=True)
def seeded():
    """The same values whatever ran before."""
    torch.manual_seed(5)


DIMS = {"gdn": (128, 128), "kda": (128, 128), "mamba2": (128, 64)}


def make_state(form, rule, batch, d_k, d_v):
    vbar = torch.randn(H, d_v, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    if form == "h16":
        return binding.ShallowState16(rule, batch, H, d_k, d_v, R, W, vbar)
    if form == "scheduled":
        return binding.ScheduledState(rule, batch, H, d_k, d_v, R, W, 0, vbar, [0] * batch)
    return binding.ShallowState(rule, batch, H, d_k, d_v, R, W, vbar, lazy=form == "lazy")


def tensors(st):
    return {k: v for k, v in vars(st).items() if isinstance(v, torch.Tensor)}


def prompt(rule, offsets, dtype, seed):
    d_k, d_v = DIMS[rule]
    x = inputs(rule, offsets[-1], H, H, d_k, d_v, len(offsets) - 1, dtype, seed, initial=False)
    return x, torch.tensor(offsets, dtype=torch.int32, device="cuda")


def args(x):
    return x["q"], x["k"], x["v"], x["g"], x["beta"]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("form", ["fp32", "lazy", "h16", "scheduled"])
def test_serving(rule, form):
    """Prompts of 1, 7, 0 and R tokens, then W - 1 decode steps, every
    read-out normed: against the dense recurrence in 64 bits."""
    offsets = [0, 1, 8, 8, 8 + R]
    B = len(offsets) - 1
    d_k, d_v = DIMS[rule]
    x, cu = prompt(rule, offsets, torch.bfloat16, 21)
    st = make_state(form, rule, B, d_k, d_v)
    o = torch.empty_like(x["v"])
    S = st.prefill(*args(x), o, cu_seqlens=cu)
    h = host(x)
    want_o, want_S = oseq.scan(rule, *(h[k] for k in ("q", "k", "v", "g", "beta")),
                               np.zeros((B, H, d_k, d_v)), offsets)
    check(o, want_o, offsets, "o")
    check(S, want_S, [0], "S")
    weight = 1 + 0.1 * torch.randn(d_v, device="cuda")
    gate = torch.randn_like(x["v"])
    y = torch.empty_like(o)
    sequence.seed_group_norm(o, y, weight=weight, gate=gate)
    flags = {"eps": 1e-5, "centered": False, "activation": "silu", "gate_first": False}
    close(y, oseq.group_norm(f64(o), f64(gate), f64(weight), None, **flags), "y")

    base = TOL_STATE_COMPRESS + (np.sqrt(R) * 2.0 ** -10 if form == "h16" else 0.0)
    read = torch.empty(B, H, d_v, device="cuda")
    z = torch.randn(B, H, d_v, device="cuda").to(torch.bfloat16)
    y = torch.empty_like(z)
    ref = f64(S)
    size = 0.0
    for t in range(W - 1):
        step = inputs(rule, B, H, H, d_k, d_v, B, torch.bfloat16, 100 + t, initial=False)
        st.step(*args(step), read)
        hs = host(step)
        each = [oseq.scan(rule, *(None if hs[k] is None else hs[k][b:b + 1]
                                  for k in ("q", "k", "v", "g", "beta")), ref[b:b + 1], [0, 1])
                for b in range(B)]
        ref = np.concatenate([s for _, s in each])
        want = np.concatenate([r for r, _ in each])
        # the state before the step was off by a share of its largest norm yet
        size = max(size, np.sqrt((ref ** 2).sum((2, 3))).max())
        err = np.sqrt(((f64(read) - want) ** 2).sum(-1)).max()
        assert err <= (base + (t + 1) * TOL_STATE_STEP) * size, (t, err, size)
        sequence.seed_group_norm(read, y, weight=weight, gate=z)
        close(y, oseq.group_norm(f64(read), f64(z), f64(weight), None, **flags), "y")


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("form", ["fp32", "lazy", "h16", "scheduled"])
def test_prefill_is_scan_and_conversion(rule, form):
    """Long prompts in two pieces, packed and padded, on another stream and
    from a graph: the bits of seed_scan and from_dense one after the other."""
    d_k, d_v = DIMS[rule]
    T, B = 150, 2
    x, cu = prompt(rule, [0, T, 2 * T], torch.bfloat16, 22)
    o1, o2 = torch.empty_like(x["v"]), torch.empty_like(x["v"])
    S = torch.empty(B, H, d_k, d_v, device="cuda")
    sequence.seed_scan(rule, *args(x), o1, S, cu_seqlens=cu)
    ref = make_state(form, rule, B, d_k, d_v)
    ref.from_dense(S)

    def same(st, other=ref):
        a, b = tensors(st), tensors(other)
        return all(torch.equal(a[k], b[k]) for k in a)

    padded = {k: None if v is None else v.view(B, T, *v.shape[1:]) for k, v in x.items()}
    st = make_state(form, rule, B, d_k, d_v)
    ws = sequence.scan_workspace(rule, padded["q"], padded["v"], B)
    got = st.prefill(*args(padded), o2.view(B, T, H, d_v), workspace=ws)
    assert torch.equal(got, S) and torch.equal(o1, o2) and same(st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st = make_state(form, rule, B, d_k, d_v)
    torch.cuda.synchronize()
    got = st.prefill(*args(x), o2, cu_seqlens=cu, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, S) and torch.equal(o1, o2) and same(st)
    st = make_state(form, rule, B, d_k, d_v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = st.prefill(*args(x), o2, cu_seqlens=cu)
    for _ in range(3):
        for t in (*tensors(st).values(), got, o2):
            if t is not st.vbar and t.is_floating_point():
                t.zero_()
        eager = make_state(form, rule, B, d_k, d_v)
        eager.prefill(*args(x), o2.clone(), cu_seqlens=cu)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, S) and torch.equal(o1, o2) and same(st) and same(eager)
    # the second prompt continues the first, from its dense state
    st = make_state(form, rule, B, d_k, d_v)
    again = st.prefill(*args(x), o2, S0=S, cu_seqlens=cu)
    both = torch.empty_like(S)
    sequence.seed_scan(rule, *args(x), o1, both, S0=S, cu_seqlens=cu)
    assert torch.equal(again, both) and torch.equal(o1, o2)


def test_prefill_refusals():
    x, cu = prompt("gdn", [0, 3, 5], torch.bfloat16, 23)
    st = make_state("fp32", "gdn", 3, 128, 128)   # three requests, two prompts
    before = {k: v.clone() for k, v in tensors(st).items()}
    with pytest.raises(ValueError, match="S has shape"):
        st.prefill(*args(x), torch.empty_like(x["v"]), cu_seqlens=cu)
    st2 = make_state("fp32", "kda", 2, 128, 128)  # another rule's gates
    with pytest.raises(ValueError, match="g has shape"):
        st2.prefill(*args(x), torch.empty_like(x["v"]), cu_seqlens=cu)
    assert st.r == 0 and all(torch.equal(before[k], v) for k, v in tensors(st).items())


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_layer(rule, dtype):
    """loss = <dy, norm(scan(...))>: each pass back against the formulas in 64
    bits from the very values it was given.

    dq and dk are sums of (do_t.u_s) k_s and (do_t.u_s) q_t.  The sequence of
    one token has the single term dk = q (do.u), and the norm's gradient do is
    at right angles to the normed read-out, which u is part of: the inner
    product of d_v terms may fall far below the size |do| |u| / sqrt(d_v) of
    unrelated ones, to which its error belongs (as for gates and write
    strengths, test_gpu_scan.py; with other values a dk of 8.5e-4 was off by
    4.2e-7).  That size times the largest entry of k or q is their scale,
    |v| standing for |u|."""
    offsets = [0, 70, 71, 200]
    d_k, d_v = DIMS[rule]
    x = inputs(rule, offsets[-1], H, 1, d_k, d_v, 3, dtype, 24)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    weight = 1 + 0.1 * torch.randn(H, d_v, device="cuda")
    gate, dy = torch.randn_like(x["v"]), torch.randn_like(x["v"])
    flags = {"eps": 1e-5, "centered": False, "activation": "silu", "gate_first": False}
    got = layer(rule, x, cu, weight, gate, dy, flags)
    h = host(x)
    norm = oseq.group_norm(f64(got["o"]), f64(gate), f64(weight), None, **flags, dy=f64(dy))
    close(got["do"], norm["x"], "do", norm.get("x_scale"))
    close(got["gate"], norm["gate"], "gate", norm.get("gate_scale"))
    want = oseq.scan_backward(rule, *(h[k] for k in ("q", "k", "v", "g", "beta", "S0")), offsets,
                              f64(got["do"]), np.zeros(x["S0"].shape))
    size = np.linalg.norm(f64(got["do"]), axis=-1) * np.linalg.norm(h["v"], axis=-1).max() / np.sqrt(d_v)
    size = size.max(1, keepdims=True)
    want["q_scale"], want["k_scale"] = size * np.abs(h["k"]).max(), size * np.abs(h["q"]).max()
    for name in ("q", "k", "v", "g", "beta", "S0"):
        if x[name] is not None:
            check(got[name], want[name], [0] if name == "S0" else offsets, name,
                  terms=want.get(name + "_scale"))


@pytest.mark.parametrize("rule", RULES)
def test_training_layer_differences(rule):
    """The layer's gradients along a random direction against central
    differences of the layer in 64 bits.  A read-out off by F32 of its unit's
    largest value, some four times its root mean square, turns the normed
    vector and with it everything behind by 4 F32; with the passes' own errors
    16 F32 of the gradients' norms bounds it.  The differences' own error is
    the third derivative's, h^2 = 1e-8 of the value."""
    offsets = [0, 70, 71, 140]
    d_k, d_v = DIMS[rule]
    x = inputs(rule, offsets[-1], H, 1, d_k, d_v, 3, torch.float32, 25)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    weight = 1 + 0.1 * torch.randn(H, d_v, device="cuda")
    gate, dy = torch.randn_like(x["v"]), torch.randn_like(x["v"])
    flags = {"eps": 1e-5, "centered": False, "activation": "silu", "gate_first": False}
    got = layer(rule, x, cu, weight, gate, dy, flags)
    names = [k for k in ("q", "k", "v", "g", "beta", "S0") if x[k] is not None] + ["gate", "weight"]
    at = {**host(x), "gate": f64(gate), "weight": f64(weight)}
    rng = np.random.default_rng(7)
    along = {k: rng.standard_normal(at[k].shape) for k in names}
    along = {k: v / np.linalg.norm(v) for k, v in along.items()}

    def loss(h):
        y = {k: v if k not in along else v + h * along[k] for k, v in at.items()}
        o, _ = oseq.scan(rule, *(y[k] for k in ("q", "k", "v", "g", "beta", "S0")), offsets)
        return (oseq.group_norm(o, y["gate"], y["weight"], None, **flags) * f64(dy)).sum()

    h = 1e-4
    want = (loss(h) - loss(-h)) / (2 * h)
    value = sum((f64(got[k]) * along[k]).sum() for k in names)
    size = sum(np.linalg.norm(f64(got[k])) for k in names)
    assert abs(value - want) <= 16 * F32 * size, (value, want, size)


def layer(rule, x, cu, weight, gate, dy, flags):
    """One layer forward and back through the kernels."""
    o, y, do = (torch.empty_like(x["v"]) for _ in range(3))
    S = torch.empty_like(x["S0"])
    sequence.seed_scan(rule, *args(x), o, S, S0=x["S0"], cu_seqlens=cu)
    sequence.seed_group_norm(o, y, weight=weight, gate=gate, **flags)
    out = {k: torch.empty_like(v) for k, v in x.items() if v is not None}
    out.update(o=o, do=do, gate=torch.empty_like(gate), weight=torch.empty_like(weight))
    sequence.seed_group_norm_backward(dy, o, do, dgate=out["gate"], dweight=out["weight"],
                                      weight=weight, gate=gate, **flags)
    sequence.seed_scan_backward(rule, *args(x), do, out["q"], out["k"], out["v"], out["g"],
                                out.get("beta"), S0=x["S0"], dS0=out["S0"], cu_seqlens=cu)
    return out
