"""Cases of the operators on channels: the short causal convolution in front of a recurrence and the selective state
space scan, each over whole sequences, backward, and for single tokens.

Each case has a plain form in elementary torch operations, the calls a user of the framework makes (`own`), and the
definition in 64 bits (`exact`).  Batches and widths follow `sink_rank_recurrent_amd/workloads.py` and
`perf/operators.py`: 64 prompts of 512 tokens, 16 or 32 heads of 128 channels, 24 ragged prompts, 4 x 2048 tokens of
training, decode steps of 64 and 256 requests.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MAX_CONV_VALUES = 1 << 26          # tokens times channels of the largest listed convolution
MAX_SELECT_VALUES = 1 << 24        # tokens times channels of a drawn scan (1 << 22 backward), 16 states a channel
MAX_STEP_VALUES = 1 << 21          # requests times channels of the largest listed step


def listed():
    return [
        # the convolution of one short prompt: the latency of a first token, 16 heads of 128 channels
        {"name": "conv_short", "op": "conv", "dtype": "bf16", "n_seq": 1, "tokens": 33, "channels": 2048, "width": 4,
         "row": 2048, "activation": "silu", "bias": False, "ragged": False, "initial": False},
        # a served layer's keys, 64 requests of 512 tokens: a slice of the rows that one projection of q, k and v made
        {"name": "conv_prefill", "op": "conv", "dtype": "bf16", "n_seq": 64, "tokens": 32768, "channels": 2048, "width": 4,
         "row": 6144, "activation": "silu", "bias": False, "ragged": False, "initial": False},
        # one layer's backward pass in training: 4 sequences of 2048 tokens
        {"name": "conv_train", "op": "conv_backward", "dtype": "bf16", "n_seq": 4, "tokens": 8192, "channels": 4096,
         "width": 4, "row": 4096, "activation": "silu", "bias": True, "ragged": False, "initial": False},
        # training on packed documents that continue earlier parts, float32, an odd number of channels
        {"name": "conv_train_ragged", "op": "conv_backward", "dtype": "f32", "n_seq": 5, "tokens": 3001, "channels": 2047,
         "width": 3, "row": 2047, "activation": "silu", "bias": True, "ragged": True, "initial": True},
        # one decode step of 64 requests
        {"name": "conv_step", "op": "conv_step", "dtype": "bf16", "batch": 64, "channels": 2048, "width": 4, "row": 6144,
         "activation": "silu", "bias": False},
        # one decode step of 256 requests, wide layer
        {"name": "conv_step_many", "op": "conv_step", "dtype": "f32", "batch": 256, "channels": 8192, "width": 4,
         "row": 8192, "activation": "silu", "bias": True},
        # prompts of every length packed behind each other, continuing from the states of an earlier part
        {"name": "select_ragged", "op": "select", "dtype": "bf16", "n_seq": 24, "tokens": 7919, "channels": 4096,
         "groups": 1, "d_state": 16, "row": 8192, "gate": True, "skip": True, "softplus": True, "ragged": True,
         "initial": True},
        # one long document, float32: the long axis is most of the parallelism there is
        {"name": "select_long", "op": "select", "dtype": "f32", "n_seq": 1, "tokens": 16384, "channels": 2048, "groups": 1,
         "d_state": 16, "row": 2048, "gate": False, "skip": True, "softplus": True, "ragged": False, "initial": False},
        # one layer's backward pass in training: 4 sequences of 2048 tokens, gated
        {"name": "select_train", "op": "select_backward", "dtype": "bf16", "n_seq": 4, "tokens": 8192, "channels": 4096,
         "groups": 1, "d_state": 16, "row": 8192, "gate": True, "skip": True, "softplus": True, "ragged": False,
         "initial": False},
        # training on packed documents in float32, two groups of an odd number of channels, few states each
        {"name": "select_train_ragged", "op": "select_backward", "dtype": "f32", "n_seq": 5, "tokens": 3001,
         "channels": 2050, "groups": 2, "d_state": 8, "row": 2050, "gate": False, "skip": True, "softplus": True,
         "ragged": True, "initial": True},
        # one decode step of 64 requests
        {"name": "select_step", "op": "select_step", "dtype": "bf16", "batch": 64, "channels": 4096, "groups": 1,
         "d_state": 16, "row": 8192, "gate": True, "skip": True, "softplus": True},
        # one decode step of 256 requests, wide layer: 134 MB of states
        {"name": "select_step_many", "op": "select_step", "dtype": "bf16", "batch": 256, "channels": 8192, "groups": 1,
         "d_state": 16, "row": 16384, "gate": True, "skip": True, "softplus": True},
    ]


def _log(rng, low, high):
    """A whole number, its logarithm spread evenly."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def _sequences(rng, most):
    tokens = _log(rng, 1, max(1, most))
    n_seq = _log(rng, 1, max(1, min(64, tokens)))
    ragged = rng.random() < 0.6
    if not ragged:
        tokens -= tokens % n_seq
    return {"n_seq": n_seq, "tokens": tokens, "ragged": ragged, "initial": rng.random() < 0.5}


def draw(rng):
    op = rng.choice(("conv", "conv_backward", "conv_step", "select", "select_backward", "select_step"))
    case = {"op": op, "dtype": rng.choice(("bf16", "bf16", "f32"))}
    channels = _log(rng, 1, 8192)
    if rng.random() < 0.5:
        channels = -(-channels // 64) * 64
    if op.startswith("conv"):
        case.update(channels=channels, width=rng.choice((2, 3, 4)), activation=rng.choice(("silu", "silu", "none")),
                    bias=rng.random() < 0.5, row=channels if rng.random() < 0.5 else 3 * channels)
        if op == "conv_step":
            case["batch"] = _log(rng, 1, min(1024, MAX_STEP_VALUES // channels))
        else:
            most = MAX_CONV_VALUES // ((1 if op == "conv" else 2) * (2 if case["dtype"] == "f32" else 1))
            case.update(_sequences(rng, min(32768, most // channels)))
        return case
    d_state = rng.choice((16, 16, 16, 8, 5, 32, 64))
    groups = rng.choice([g for g in (1, 1, 2, 4) if channels % g == 0])
    case.update(channels=channels, groups=groups, d_state=d_state, gate=rng.random() < 0.5, skip=rng.random() < 0.7,
                softplus=rng.random() < 0.7, row=channels if rng.random() < 0.5 else 2 * channels)
    padded = channels * max(1.0, d_state / 16)
    if op == "select_step":
        case["batch"] = _log(rng, 1, min(1024, int(MAX_STEP_VALUES / padded)))
    else:
        most = MAX_SELECT_VALUES if op == "select" else MAX_SELECT_VALUES // 4
        case.update(_sequences(rng, min(8192, int(most / padded))))
    return case


def lengths(case):
    """The sequences' lengths: equal ones, or (ragged) very different ones, an empty one among them where there are three."""
    n, tokens = case["n_seq"], case["tokens"]
    if not case["ragged"]:
        return [tokens // n] * n
    weights = [1.0 + (7 * i) % n for i in range(n)]
    if n >= 3:
        weights[1] = 0.0
    out = [int(tokens * w / sum(weights)) for w in weights]
    out[0] += tokens - sum(out)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, dt, channels = case["op"], DTYPES[case["dtype"]], case["channels"]
    step = op.endswith("step")

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case, "workspace": None}
    rows = case["batch"] if step else case["tokens"]
    n = case["batch"] if step else case["n_seq"]
    if not step:
        lens = lengths(case)
        s["max_len"] = max(lens)
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    empty = {"device": "cuda", "dtype": dt}
    if op.startswith("conv"):
        K = case["width"]
        # a slice of the projection's rows
        at = case["row"] - channels
        s["x"] = normal(rows, case["row"]).to(dt)[:, at // 2:at // 2 + channels]
        s["weight"] = (2 * uniform(channels, K) - 1) / math.sqrt(K)
        s["bias"] = 0.2 * normal(channels) if case["bias"] else None
        s["S0"] = normal(n, K - 1, channels).to(dt) if step or case["initial"] else None
        if op == "conv_backward":
            s["dy"] = (0.02 * normal(rows, channels)).to(dt)
            s["dS"] = (0.02 * normal(n, K - 1, channels)).to(dt) if case["initial"] else None
            s["out"] = {"dx": torch.empty(rows, channels, **empty), "dweight": torch.empty_like(s["weight"])}
            if s["bias"] is not None:
                s["out"]["dbias"] = torch.empty_like(s["bias"])
            if s["S0"] is not None:
                s["out"]["dS0"] = torch.empty_like(s["S0"])
        else:
            s["y"] = torch.empty(rows, channels, **empty)
            s["S"] = torch.empty(n, K - 1, channels, **empty)
        return s
    G, N = case["groups"], case["d_state"]
    # x and its gate are halves of one projection's rows where these are wider; x went through a convolution and SiLU
    xz = normal(rows, max(case["row"], channels * (2 if case["gate"] else 1)))
    xz[:, :channels] *= torch.sigmoid(xz[:, :channels])
    xz = xz.to(dt)
    s["x"] = xz[:, :channels]
    s["z"] = xz[:, channels:2 * channels] if case["gate"] else None
    # steps between 0.001 and 0.1, their logarithm spread evenly over the channels, moved by the token
    steps = torch.exp(uniform(channels) * math.log(100.0) + math.log(0.001))
    if case["softplus"]:
        s["dt"] = (0.5 * normal(rows, channels)).to(dt)
        s["dt_bias"] = steps + torch.log(-torch.expm1(-steps))
    else:
        s["dt"] = (steps * torch.exp(0.5 * normal(rows, channels))).to(dt)
        s["dt_bias"] = None
    # rates 1 .. d_state, as trained layers start from, moved by training
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.2 * normal(channels, N))
    # B and C lie behind each other in the rows of one projection
    bc = normal(rows, 2, G, N).to(dt)
    s["B"], s["C"] = bc[:, 0], bc[:, 1]
    s["D"] = 1 + 0.1 * normal(channels) if case["skip"] else None
    s["S0"] = 0.3 * normal(n, channels, N) if step or case["initial"] else None
    if op == "select_backward":
        s["dy"] = (0.02 * normal(rows, channels)).to(dt)
        s["dS"] = 0.02 * normal(n, channels, N) if case["initial"] else None
        out = {"dx": torch.empty(rows, channels, **empty), "ddt": torch.empty(rows, channels, **empty),
               "dA": torch.empty_like(s["A"]), "dB": torch.empty(rows, G, N, **empty), "dC": torch.empty(rows, G, N, **empty)}
        for name, like in (("dD", "D"), ("ddt_bias", "dt_bias"), ("dS0", "S0")):
            if s[like] is not None:
                out[name] = torch.empty_like(s[like])
        if s["z"] is not None:
            out["dz"] = torch.empty(rows, channels, **empty)
        s["out"] = out
    else:
        s["y"] = torch.empty(rows, channels, **empty)
        s["S"] = torch.empty(n, channels, N, device="cuda")
    return s


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    step = case["op"].endswith("step")
    rows, n, ch = (case["batch"] if step else case["tokens"]), (case["batch"] if step else case["n_seq"]), case["channels"]
    initial = step or case["initial"]
    if case["op"].startswith("conv"):
        K = case["width"]
        weights = 4 * ch * (K + (1 if case["bias"] else 0))
        state = e * n * (K - 1) * ch
        if case["op"] == "conv_backward":     # x, dy in, dx out; weights in, their gradients out; the states' likewise
            return {"bytes": 3 * e * rows * ch + 2 * weights + (3 * state if initial else 0),
                    "flops": float(rows * ch * (6 * K + 12))}
        return {"bytes": 2 * e * rows * ch + weights + state * (2 if initial else 1), "flops": float(rows * ch * (2 * K + 5))}
    N, G = case["d_state"], case["groups"]
    tokens = e * rows * (ch * (3 if case["gate"] else 2) + 2 * G * N)
    weights = 4 * ch * (N + (1 if case["skip"] else 0) + (1 if case["softplus"] else 0))
    state = 4 * n * ch * N
    # a state's update and read-out: the rate times the step, its exponential, the input, two multiply-adds
    flops = 7.0 * rows * ch * N
    if case["op"] == "select_backward":
        return {"bytes": 2 * tokens + e * rows * ch + 2 * weights + (3 * state if initial else 0), "flops": 3 * flops}
    return {"bytes": tokens + e * rows * ch + weights + state * (2 if initial else 1), "flops": flops}


# ---------------------------------------------------------------- the plain forms

def _plain_conv(case, x, weight, bias, S0, cu):
    """y before its rounding, and the last states: taps gathered from the inputs behind the first states."""
    K, channels = weight.shape[1], weight.shape[0]
    n, tokens = cu.shape[0] - 1, x.shape[0]
    first = torch.zeros(n, K - 1, channels, device=x.device) if S0 is None else S0.float()
    rows = torch.cat((first.reshape(n * (K - 1), channels), x.float()))
    held = n * (K - 1)
    start = cu[:-1].long()
    of = torch.searchsorted(cu[1:].contiguous(), torch.arange(tokens, device=x.device, dtype=cu.dtype), right=True)

    def taken(at, s):
        """Row of token `at` of sequence s, or of its first state where `at` lies before it."""
        before = s * (K - 1) + (K - 1) + at - start[s]
        return torch.where(at >= start[s], held + at, before)

    y = torch.zeros(tokens, channels, device=x.device)
    for j in range(K):
        y = y + rows[taken(torch.arange(tokens, device=x.device) - (K - 1) + j, of)] * weight[:, j]
    if bias is not None:
        y = y + bias
    if case["activation"] == "silu":
        y = y * torch.sigmoid(y)
    last = cu[1:, None].long() - (K - 1) + torch.arange(K - 1, device=x.device)
    return y, rows[taken(last, torch.arange(n, device=x.device)[:, None])]


def _steps_of(dt, dt_bias, softplus):
    v = dt.float()
    if dt_bias is not None:
        v = v + dt_bias
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v))) if softplus else v


def _gated(y, x, D, z):
    if D is not None:
        y = y + D * x.float()
    if z is not None:
        z = z.float()
        y = y * (z * torch.sigmoid(z))
    return y


def _plain_select(case, x, dt, A, B, C, D, z, dt_bias, S, cu, max_len):
    """64 tokens of every part side by side from a state of zero, the states carried from part to part, then what
    they add to the parts' read-outs."""
    L = 64
    M = max(1, -(-max_len // L))
    n, G, N, channels = cu.shape[0] - 1, case["groups"], case["d_state"], case["channels"]
    start, end = cu[:-1].long(), cu[1:].long()
    at = start[:, None] + torch.arange(M * L, device=x.device)
    real = at < end[:, None]
    at = at.clamp(max=x.shape[0] - 1)

    def parts(rows):
        """[tokens, ...] as [n, M, L, ...], zero behind each sequence's end."""
        keep = real.reshape(real.shape + (1,) * (rows.dim() - 1))
        return torch.where(keep, rows[at], torch.zeros((), device=x.device)).reshape((n, M, L) + rows.shape[1:])

    step = _steps_of(dt, dt_bias, case["softplus"])
    delta = parts(step).reshape(n, M, L, G, channels // G)
    put = parts(step * x.float()).reshape(n, M, L, G, channels // G)
    B, C = parts(B.float())[:, :, :, :, None], parts(C.float())[:, :, :, :, None]
    A = A.reshape(G, channels // G, N)
    gone = torch.cumsum(delta, 2)
    h = torch.zeros(n, M, G, channels // G, N, device=x.device)
    local = []
    for j in range(L):
        h = torch.exp(delta[:, :, j, ..., None] * A) * h + put[:, :, j, ..., None] * B[:, :, j]
        local.append((h * C[:, :, j]).sum(-1))
    S = torch.zeros(n, channels, N, device=x.device) if S is None else S
    S = S.reshape(n, G, channels // G, N)
    starts = []
    for m in range(M):
        starts.append(S)
        S = torch.exp(gone[:, m, -1, ..., None] * A) * S + h[:, m]
    first = torch.stack(starts, 1)
    y = torch.stack([local[j] + (torch.exp(gone[:, :, j, ..., None] * A) * first * C[:, :, j]).sum(-1) for j in range(L)], 2)
    y = y.reshape(n, M * L, channels)[real]
    return _gated(y, x, D, z), S.reshape(n, channels, N)


def _plain_conv_step(case, x, weight, bias, S0):
    rows = torch.cat((S0.float(), x.float()[:, None]), 1)
    y = (rows * weight.t()).sum(1)
    if bias is not None:
        y = y + bias
    if case["activation"] == "silu":
        y = y * torch.sigmoid(y)
    return y, rows[:, 1:]


def _plain_select_step(case, x, dt, A, B, C, D, z, dt_bias, S0):
    each = case["channels"] // case["groups"]
    step = _steps_of(dt, dt_bias, case["softplus"])
    B, C = B.float().repeat_interleave(each, 1), C.float().repeat_interleave(each, 1)
    S = torch.exp(step[..., None] * A) * S0 + (step * x.float())[..., None] * B
    return _gated((S * C).sum(-1), x, D, z), S


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    act = s["x"].dtype
    if op == "conv_step":
        y, S = _plain_conv_step(case, s["x"], s["weight"], s["bias"], s["S0"])
        return {"y": y.to(act), "S": S.to(act)}
    if op == "select_step":
        y, S = _plain_select_step(case, *(s[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0")))
        return {"y": y.to(act), "S": S}
    if op.startswith("conv"):
        names = ("x", "weight", "bias", "S0")

        def forward(a):
            return _plain_conv(case, a["x"], a["weight"], a["bias"], a["S0"], s["cu"])
    else:
        names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0")

        def forward(a):
            return _plain_select(case, *(a[k] for k in names), s["cu"], s["max_len"])
    if not op.endswith("backward"):
        y, S = forward(s)
        return {"y": y.to(act), "S": S.to(s["S"].dtype)}
    # in 32 bits throughout: each gradient is rounded once, at the end
    leaves = {k: s[k].detach().float().clone().requires_grad_() for k in names if s[k] is not None}
    y, S = forward({k: leaves.get(k) for k in names})
    outs, grads = [y], [s["dy"].float()]
    if s["dS"] is not None:
        outs, grads = outs + [S], grads + [s["dS"].float()]
    got = torch.autograd.grad(outs, list(leaves.values()), grads)
    return {"d" + k: g.to(s[k].dtype) for k, g in zip(leaves, got)}


def _own(s, case, op):
    from sink_rank_recurrent_amd import channels
    if op.startswith("conv"):
        flags = {"bias": s["bias"], "activation": None if case["activation"] == "none" else case["activation"], "S0": s["S0"]}
        if op == "conv_step":
            channels.seed_short_conv_step(s["x"], s["weight"], s["y"], s["S"], **flags)
        elif op == "conv":
            channels.seed_short_conv(s["x"], s["weight"], s["y"], S=s["S"], cu_seqlens=s["cu"], **flags)
        else:
            if s["workspace"] is None:
                s["workspace"] = channels.short_conv_workspace(s["x"], s["weight"], case["n_seq"])
            out = s["out"]
            channels.seed_short_conv_backward(s["dy"], s["x"], s["weight"], out["dx"], dweight=out["dweight"],
                                              dbias=out.get("dbias"), dS=s["dS"], dS0=out.get("dS0"),
                                              cu_seqlens=s["cu"], workspace=s["workspace"], **flags)
            return out
        return {"y": s["y"], "S": s["S"]}
    inputs = [s[k] for k in ("x", "dt", "A", "B", "C")]
    flags = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "softplus": case["softplus"], "S0": s["S0"]}
    if op == "select_step":
        channels.seed_selective_step(*inputs, s["y"], s["S"], **flags)
        return {"y": s["y"], "S": s["S"]}
    if s["workspace"] is None:      # made once for a state, as a program that runs many steps keeps it
        s["workspace"] = channels.selective_scan_workspace(s["x"], s["B"], case["n_seq"], backward=op != "select")
    flags.update(cu_seqlens=s["cu"], workspace=s["workspace"])
    if op == "select":
        channels.seed_selective_scan(*inputs, s["y"], s["S"], **flags)
        return {"y": s["y"], "S": s["S"]}
    out = s["out"]
    channels.seed_selective_scan_backward(s["dy"], *inputs, out["dx"], out["ddt"], out["dA"], out["dB"], out["dC"],
                                          dD=out.get("dD"), dz=out.get("dz"), ddt_bias=out.get("ddt_bias"),
                                          dS=s["dS"], dS0=out.get("dS0"), **flags)
    return out


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.endswith("step"):                # a step is a sequence of one token
        rows = case["batch"]
        s["cu"] = torch.arange(rows + 1, device="cuda", dtype=torch.int32)
    if op.startswith("conv"):
        return _conv64(s, case, op == "conv_backward")
    return _select64_back(s, case) if op == "select_backward" else _select64(s, case)[0]


def _conv64(s, case, backward):
    """Sequence by sequence, the first state in front of the inputs."""
    x, w, cu = s["x"].double(), s["weight"].double(), s["cu"].tolist()
    K, channels, n = w.shape[1], w.shape[0], len(cu) - 1
    silu = case["activation"] == "silu"
    y, S = torch.zeros_like(x), torch.zeros(n, K - 1, channels, device="cuda", dtype=torch.float64)
    d = {"dx": torch.zeros_like(x), "dweight": torch.zeros_like(w), "dS0": torch.zeros_like(S)}
    dbias = torch.zeros(channels, device="cuda", dtype=torch.float64)
    for i in range(n):
        a, b = cu[i], cu[i + 1]
        held = torch.zeros(K - 1, channels, device="cuda", dtype=torch.float64) if s["S0"] is None else s["S0"][i].double()
        line = torch.cat((held, x[a:b]))
        S[i] = line[b - a:]
        pre = sum(line[j:j + b - a] * w[:, j] for j in range(K))
        if s["bias"] is not None:
            pre = pre + s["bias"].double()
        sig = 1 / (1 + torch.exp(-pre))
        y[a:b] = pre * sig if silu else pre
        if not backward:
            continue
        dpre = s["dy"][a:b].double()
        if silu:
            dpre = dpre * sig * (1 + pre * (1 - sig))
        dline = torch.zeros_like(line)
        if s["dS"] is not None:
            dline[b - a:] += s["dS"][i].double()
        for j in range(K):
            dline[j:j + b - a] += dpre * w[:, j]
            d["dweight"][:, j] += (dpre * line[j:j + b - a]).sum(0)
        dbias += dpre.sum(0)
        d["dx"][a:b], d["dS0"][i] = dline[K - 1:], dline[:K - 1]
    if not backward:
        return {"y": y, "S": S}
    out = {"dx": d["dx"], "dweight": d["dweight"]}
    if s["bias"] is not None:
        out["dbias"] = dbias
    if s["S0"] is not None:
        out["dS0"] = d["dS0"]
    return out


def _inputs64(s, case):
    each = case["channels"] // case["groups"]
    q = {k: None if s[k] is None else s[k].double() for k in ("x", "dt", "A", "D", "z", "dt_bias")}
    q["B"], q["C"] = (s[k].double().repeat_interleave(each, 1) for k in ("B", "C"))
    v = q["dt"] if q["dt_bias"] is None else q["dt"] + q["dt_bias"]
    # log(1 + e^v) without overflow; its slope
    q["step"] = torch.logaddexp(v, torch.zeros_like(v)) if case["softplus"] else v
    q["slope"] = 1 / (1 + torch.exp(-v)) if case["softplus"] else torch.ones_like(v)
    # the sequences by falling length: those that still run are a prefix
    cu = s["cu"].tolist()
    order = sorted(range(len(cu) - 1), key=lambda i: cu[i] - cu[i + 1])
    live = [cu[i + 1] - cu[i] for i in order]
    return q, order, torch.tensor([cu[i] for i in order], device="cuda"), live


def _select64(s, case, keep=False):
    """The recurrence as it is defined, a token of every sequence at a time; (keep) the state behind each token."""
    q, order, starts, live = _inputs64(s, case)
    n, N, channels = len(order), case["d_state"], case["channels"]
    S = torch.zeros(n, channels, N, device="cuda", dtype=torch.float64) if s["S0"] is None else s["S0"].double()[order]
    h0 = S.clone()
    read = torch.zeros_like(q["x"])
    states = torch.zeros(q["x"].shape + (N,), device="cuda", dtype=torch.float64) if keep else None
    for t in range(live[0]):
        m = sum(length > t for length in live)
        at = starts[:m] + t
        step = q["step"][at][..., None]
        S[:m] = torch.exp(step * q["A"]) * S[:m] + step * q["x"][at][..., None] * q["B"][at]
        read[at] = (S[:m] * q["C"][at]).sum(-1)
        if keep:
            states[at] = S[:m]
    y = read if q["D"] is None else read + q["D"] * q["x"]
    ungated = y
    if q["z"] is not None:
        y = y * q["z"] / (1 + torch.exp(-q["z"]))
    out = torch.empty_like(S)
    out[order] = S
    return {"y": y, "S": out}, q, order, starts, live, h0, states, ungated


def _select64_back(s, case):
    """The chain rule through each token, the last one first."""
    _, q, order, starts, live, h0, states, ungated = _select64(s, case, keep=True)
    each, channels, N = case["channels"] // case["groups"], case["channels"], case["d_state"]
    d = s["dy"].double()
    out = {}
    if q["z"] is not None:
        sig = 1 / (1 + torch.exp(-q["z"]))
        out["dz"] = d * ungated * sig * (1 + q["z"] * (1 - sig))
        d = d * q["z"] * sig
    G = torch.zeros_like(h0) if s["dS"] is None else s["dS"].double()[order]
    dx, dstep = torch.zeros_like(q["x"]), torch.zeros_like(q["x"])
    dA = torch.zeros_like(q["A"])
    # rows of gradients for B and C, summed over a group's channels as they come
    dB = torch.zeros(q["x"].shape[0], case["groups"], N, device="cuda", dtype=torch.float64)
    dC = torch.zeros_like(dB)
    for t in reversed(range(live[0])):
        m = sum(length > t for length in live)
        at = starts[:m] + t
        step, x = q["step"][at][..., None], q["x"][at][..., None]
        decay = torch.exp(step * q["A"])
        before = states[at - 1] if t else h0[:m]
        G[:m] += d[at][..., None] * q["C"][at]
        now = G[:m]
        dC[at] = (d[at][..., None] * states[at]).unflatten(1, (case["groups"], each)).sum(2)
        dB[at] = (now * step * x).unflatten(1, (case["groups"], each)).sum(2)
        put = (now * q["B"][at]).sum(-1)
        rate = now * decay * before
        dx[at] = put * q["step"][at]
        dstep[at] = put * q["x"][at] + (rate * q["A"]).sum(-1)
        dA += (rate * step).sum(0)
        G[:m] = now * decay
    if q["D"] is not None:
        dx = dx + d * q["D"]
        out["dD"] = (d * q["x"]).sum(0)
    ddt = dstep * q["slope"]
    if q["dt_bias"] is not None:
        out["ddt_bias"] = ddt.sum(0)
    if s["S0"] is not None:
        out["dS0"] = torch.empty_like(G)
        out["dS0"][order] = G
    out.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC)
    return out
