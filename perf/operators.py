"""Cases of the operators over whole sequences: the gated linear recurrence (prefill), its backward pass, and the
heads' group norm with a gate and an activation, forward and backward.

Each case has a plain form in elementary torch operations, the calls a user of the framework makes (`own`), and the
definition in 64 bits (`exact`).  The head shapes, gates and inputs follow `sink_rank_recurrent_amd/workloads.py`:
keys and queries of unit length, values around a direction of their head, Gated DeltaNet gates in 0.9 .. 0.999, Kimi
Delta Attention gates in 0.95 .. 0.9999 per key channel, Mamba-2 gates exp(-softplus(z) / 10).
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MAX_TOKEN_HEADS = 1 << 19      # tokens times heads of the largest listed recurrence
MAX_BACKWARD_TOKEN_HEADS = 1 << 17
MAX_NORM_VALUES = 1 << 26


def listed():
    return [
        # one short prompt, the latency of a first token: half a chunk of 64 tokens, 16 heads
        {"name": "prefill_short_gdn", "op": "scan", "rule": "gdn", "dtype": "bf16", "n_seq": 1, "tokens": 33, "heads": 16,
         "key_heads": 16, "d_k": 128, "d_v": 128, "ragged": False, "initial": False},
        # the prefill of a served layer: 64 requests of 512 tokens, 16 heads
        {"name": "prefill_batch_gdn", "op": "scan", "rule": "gdn", "dtype": "bf16", "n_seq": 64, "tokens": 32768, "heads": 16,
         "key_heads": 16, "d_k": 128, "d_v": 128, "ragged": False, "initial": False},
        # prompts of every length packed behind each other, continuing from the states of an earlier part
        {"name": "prefill_ragged_kda", "op": "scan", "rule": "kda", "dtype": "bf16", "n_seq": 24, "tokens": 7919, "heads": 32,
         "key_heads": 32, "d_k": 128, "d_v": 128, "ragged": True, "initial": True},
        # many narrow heads that share their keys and queries in groups of eight
        {"name": "prefill_shared_mamba2", "op": "scan", "rule": "mamba2", "dtype": "bf16", "n_seq": 8, "tokens": 8192,
         "heads": 64, "key_heads": 8, "d_k": 128, "d_v": 64, "ragged": False, "initial": False},
        # one long document, few heads, float32 inputs: the long axis is all the parallelism there is
        {"name": "prefill_long_gdn", "op": "scan", "rule": "gdn", "dtype": "f32", "n_seq": 1, "tokens": 16384, "heads": 16,
         "key_heads": 16, "d_k": 64, "d_v": 64, "ragged": False, "initial": True},
        # one layer's backward pass in training: 4 sequences of 2048 tokens
        {"name": "train_gdn", "op": "scan_backward", "rule": "gdn", "dtype": "bf16", "n_seq": 4, "tokens": 8192, "heads": 16,
         "key_heads": 16, "d_k": 128, "d_v": 128, "ragged": False, "initial": False},
        # training on packed documents, gates per key channel
        {"name": "train_ragged_kda", "op": "scan_backward", "rule": "kda", "dtype": "bf16", "n_seq": 5, "tokens": 3001,
         "heads": 16, "key_heads": 16, "d_k": 128, "d_v": 128, "ragged": True, "initial": True},
        # training in float32 with keys and queries shared by all heads of a group
        {"name": "train_shared_mamba2", "op": "scan_backward", "rule": "mamba2", "dtype": "f32", "n_seq": 2, "tokens": 2048,
         "heads": 32, "key_heads": 4, "d_k": 128, "d_v": 64, "ragged": False, "initial": False},
        # one decode step's read-outs of 64 requests x 16 heads, gated
        {"name": "norm_decode", "op": "norm", "rows": 64, "groups": 16, "d": 128, "x": "f32", "io": "bf16", "gate": "after",
         "activation": "silu", "centered": False, "shared": True, "bias": False},
        # the read-outs of a prefill, mean and variance per head, no gate
        {"name": "norm_prefill", "op": "norm", "rows": 32768, "groups": 16, "d": 128, "x": "bf16", "io": "bf16", "gate": "none",
         "activation": "silu", "centered": True, "shared": False, "bias": True},
        # training: per-head norm with the gate behind it
        {"name": "norm_train", "op": "norm_backward", "rows": 8192, "groups": 16, "d": 128, "x": "bf16", "io": "bf16",
         "gate": "after", "activation": "silu", "centered": False, "shared": True, "bias": False},
        # training: wide groups, an odd number of channels, the gate in front of the norm
        {"name": "norm_train_wide", "op": "norm_backward", "rows": 4001, "groups": 2, "d": 2047, "x": "f32", "io": "f32",
         "gate": "before", "activation": "silu", "centered": True, "shared": False, "bias": True},
    ]


def _log(rng, low, high):
    """A whole number, its logarithm spread evenly."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(("scan", "scan", "scan_backward", "norm", "norm_backward"))
    if op.startswith("scan"):
        rule = rng.choice(("gdn", "kda", "mamba2"))
        d_k, d_v = rng.choice(((128, 128), (128, 64), (64, 64)))
        heads = rng.choice((1, 3, 4, 8, 16, 24, 32))
        key_heads = rng.choice([h for h in (1, 2, 4, 8, heads) if heads % h == 0])
        most = MAX_TOKEN_HEADS if op == "scan" and rule != "kda" else MAX_BACKWARD_TOKEN_HEADS
        tokens = _log(rng, 1, min(8192, most // heads))
        n_seq = _log(rng, 1, max(1, min(32, tokens)))
        ragged = rng.random() < 0.6
        if not ragged:
            tokens -= tokens % n_seq
        return {"op": op, "rule": rule, "dtype": rng.choice(("bf16", "bf16", "f32")), "n_seq": n_seq, "tokens": tokens,
                "heads": heads, "key_heads": key_heads, "d_k": d_k, "d_v": d_v, "ragged": ragged,
                "initial": rng.random() < 0.5}
    d = _log(rng, 3, 8192)
    groups = rng.choice((1, 2, 5, 16, 32))
    rows = _log(rng, 1, max(1, min(32768, MAX_NORM_VALUES // 4 // (groups * d))))
    gate = rng.choice(("none", "after", "before"))
    return {"op": op, "rows": rows, "groups": groups, "d": d, "x": rng.choice(("f32", "bf16")),
            "io": rng.choice(("f32", "bf16")), "gate": gate, "activation": rng.choice(("silu", "sigmoid")),
            "centered": rng.random() < 0.5, "shared": rng.random() < 0.5, "bias": rng.random() < 0.5}


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

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    if case["op"].startswith("scan"):
        rule, T, H, HK = case["rule"], case["tokens"], case["heads"], case["key_heads"]
        d_k, d_v, n, dt = case["d_k"], case["d_v"], case["n_seq"], DTYPES[case["dtype"]]
        lens = lengths(case)
        s["max_len"] = max(lens)
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["q"] = torch.nn.functional.normalize(normal(T, HK, d_k), dim=-1).to(dt)
        s["k"] = torch.nn.functional.normalize(normal(T, HK, d_k), dim=-1).to(dt)
        s["v"] = (normal(1, H, d_v) + 0.3 * normal(T, H, d_v)).to(dt)
        if rule == "gdn":
            s["g"] = 0.9 + 0.099 * uniform(T, H)
        elif rule == "kda":
            s["g"] = 0.95 + 0.0499 * uniform(T, H, d_k)
        else:
            s["g"] = torch.exp(-0.1 * torch.nn.functional.softplus(normal(T, H)))
        s["beta"] = None if rule == "mamba2" else uniform(T, H)
        s["S0"] = 0.3 * normal(n, H, d_k, d_v) if case["initial"] else None
        # buffers a program keeps: the outputs, and the workspace of the call
        like = torch.empty_like
        if case["op"] == "scan":
            s["o"], s["S"] = like(s["v"]), torch.empty(n, H, d_k, d_v, device="cuda")
        else:
            s["do"] = (0.02 * normal(T, H, d_v)).to(dt)
            s["dS"] = 0.02 * normal(n, H, d_k, d_v) if case["initial"] else None
            s["out"] = {"dq": like(s["q"]), "dk": like(s["k"]), "dv": like(s["v"]), "dg": like(s["g"])}
            if s["beta"] is not None:
                s["out"]["dbeta"] = like(s["beta"])
            if case["initial"]:
                s["out"]["dS0"] = like(s["S0"])
        s["workspace"] = None
        return s
    rows, G, d = case["rows"], case["groups"], case["d"]
    xt, io = DTYPES[case["x"]], DTYPES[case["io"]]
    s["x"] = (0.5 * normal(1, G, d) + normal(rows, G, d)).to(xt)
    s["gate"] = normal(rows, G, d).to(io) if case["gate"] != "none" else None
    wshape = (d,) if case["shared"] else (G, d)
    s["weight"] = 1 + 0.2 * normal(*wshape)
    s["bias"] = 0.2 * normal(*wshape) if case["bias"] else None
    s["eps"] = 1e-5
    if case["op"] == "norm":
        s["y"] = torch.empty(rows, G, d, device="cuda", dtype=io)
    else:
        s["dy"] = (0.02 * normal(rows, G, d)).to(io)
        s["out"] = {"dx": torch.empty_like(s["x"]), "dweight": torch.empty_like(s["weight"])}
        if s["bias"] is not None:
            s["out"]["dbias"] = torch.empty_like(s["bias"])
        if s["gate"] is not None:
            s["out"]["dgate"] = torch.empty_like(s["gate"])
        s["workspace"] = None
    return s


def work(case):
    e = {"f32": 4, "bf16": 2}
    if case["op"].startswith("scan"):
        T, H, HK, d_k, d_v, n = (case[x] for x in ("tokens", "heads", "key_heads", "d_k", "d_v", "n_seq"))
        b = e[case["dtype"]]
        gates = 4 * T * H * (d_k if case["rule"] == "kda" else 1) + (0 if case["rule"] == "mamba2" else 4 * T * H)
        state = 4 * n * H * d_k * d_v
        once = b * T * (2 * HK * d_k + H * d_v) + gates + (state if case["initial"] else 0)
        # the recurrence itself, a token at a time: write, read-out and (delta rules) the look-up of the key
        flops = (6 if case["rule"] == "mamba2" else 8) * T * H * d_k * d_v
        if case["op"] == "scan":
            return {"bytes": once + b * T * H * d_v + state, "flops": flops}
        # inputs and the read-outs' gradient in, every input's gradient out
        return {"bytes": 2 * once + b * T * H * d_v + (state if case["initial"] else 0), "flops": 2.5 * flops}
    N = case["rows"] * case["groups"] * case["d"]
    w = 4 * case["d"] * (1 if case["shared"] else case["groups"]) * (2 if case["bias"] else 1)
    x, io, gate = e[case["x"]], e[case["io"]], case["gate"] != "none"
    if case["op"] == "norm":
        return {"bytes": N * (x + io * (2 if gate else 1)) + w, "flops": 12.0 * N}
    return {"bytes": N * (2 * x + io * (3 if gate else 1)) + 2 * w, "flops": 30.0 * N}


# ---------------------------------------------------------------- the plain forms

def _padded(x, cu, length):
    """x [tokens, heads, ...] as [n_seq, heads, length, ...] in 32 bits, and which rows are real."""
    start, end = cu[:-1].long(), cu[1:].long()
    at = start[:, None] + torch.arange(length, device=x.device)
    real = at < end[:, None]
    rows = x.float()[at.clamp(max=x.shape[0] - 1)]
    rows = torch.where(real.reshape(real.shape + (1,) * (x.dim() - 1)), rows, torch.zeros((), device=x.device))
    return rows.transpose(1, 2), real


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A: the finite product of (I + (-A)^(2^j))."""
    n = A.shape[-1]
    eye = torch.eye(n, device=A.device)
    power, out, size = -A, eye - A, 2
    while size < n:
        power = power @ power
        out = out + out @ power
        size *= 2
    return out


def _plain_scan(case, q, k, v, g, beta, S, cu, max_len):
    """Chunks of the sequences side by side, the state carried from chunk to chunk."""
    rule = case["rule"]
    C = 64
    N = max(1, -(-max_len // C))
    shared = case["heads"] // case["key_heads"]

    def chunks(x):
        rows, real = _padded(x, cu, N * C)
        return rows.reshape(rows.shape[:2] + (N, C) + rows.shape[3:]), real

    q, real = chunks(q)
    q, k, v = q.repeat_interleave(shared, 1), chunks(k)[0].repeat_interleave(shared, 1), chunks(v)[0]
    alive = real.reshape(real.shape[0], 1, N, C)
    g = chunks(g)[0]
    g = torch.where(alive if g.dim() == 4 else alive[..., None], g, torch.ones((), device=g.device))
    if g.dim() == 4:
        g = g[..., None]
    decay = torch.cumsum(torch.log(g.double()), 3)          # [n, H, N, C, 1 or d_k], from the chunk's first token
    P = torch.exp(decay).float()
    F = torch.exp(decay[:, :, :, -1:] - decay).float()
    lower = torch.ones(C, C, device=g.device, dtype=torch.bool).tril()
    if g.shape[-1] == 1:
        between = decay - decay.transpose(-1, -2)
        between = torch.exp(torch.where(lower, between, torch.full((), -torch.inf, device=g.device, dtype=torch.float64)).float())
        M = (q @ k.transpose(-1, -2)) * between
        L = (k @ k.transpose(-1, -2)) * between
    else:
        back = (k * torch.exp(-decay).float()).transpose(-1, -2)
        M = ((q * P) @ back).tril()
        L = (k * P) @ back
    if rule == "mamba2":
        U, W = v, None
    else:
        beta = chunks(beta)[0][..., None]
        X = _inverse((L * beta).tril(-1)) * beta.transpose(-1, -2)
        U, W = X @ v, X @ (k * P)
    Q, K, last = q * P, k * F, P[:, :, :, -1]
    if S is None:
        S = torch.zeros(q.shape[0], q.shape[1], q.shape[-1], v.shape[-1], device=q.device)
    out = []
    for c in range(N):
        u = U[:, :, c] if W is None else U[:, :, c] - W[:, :, c] @ S
        out.append(Q[:, :, c] @ S + M[:, :, c] @ u)
        S = last[:, :, c, :, None] * S + K[:, :, c].transpose(-1, -2) @ u
    o = torch.stack(out, 2).reshape(q.shape[0], q.shape[1], N * C, -1).transpose(1, 2)
    return o[real], S


def _plain_norm(case, x, gate, weight, bias, eps):
    x, act = x.float(), torch.sigmoid
    if gate is not None:
        gate = gate.float()
        gate = act(gate) * gate if case["activation"] == "silu" else act(gate)
    if case["gate"] == "before":
        x = x * gate
    if case["centered"]:
        x = x - x.mean(-1, keepdim=True)
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    if bias is not None:
        n = n + bias
    if case["gate"] == "after":
        return n * gate
    if case["gate"] == "none":
        return n * act(n) if case["activation"] == "silu" else act(n)
    return n


def run(s):
    case = s["case"]
    if own:
        from sink_rank_recurrent_amd import sequence
        if case["op"] == "scan":
            sequence.seed_scan(case["rule"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], s["S"], S0=s["S0"],
                               cu_seqlens=s["cu"], workspace=_workspace(s, False))
            return {"o": s["o"], "S": s["S"]}
        if case["op"] == "scan_backward":
            out = s["out"]
            sequence.seed_scan_backward(case["rule"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], out["dq"],
                                        out["dk"], out["dv"], out["dg"], out.get("dbeta"), S0=s["S0"], dS=s["dS"],
                                        dS0=out.get("dS0"), cu_seqlens=s["cu"], workspace=_workspace(s, True))
            return out
        flags = {"weight": s["weight"], "bias": s["bias"], "gate": s["gate"], "eps": s["eps"], "centered": case["centered"],
                 "activation": case["activation"], "gate_first": case["gate"] == "before"}
        if case["op"] == "norm":
            sequence.seed_group_norm(s["x"], s["y"], **flags)
            return {"y": s["y"]}
        out = s["out"]
        if s["workspace"] is None:
            s["workspace"] = sequence.group_norm_workspace(s["x"], s["weight"])
        sequence.seed_group_norm_backward(s["dy"], s["x"], out["dx"], dgate=out.get("dgate"), dweight=out["dweight"],
                                          dbias=out.get("dbias"), workspace=s["workspace"], **flags)
        return out
    if case["op"] == "scan":
        o, S = _plain_scan(case, s["q"], s["k"], s["v"], s["g"], s["beta"], s["S0"], s["cu"], s["max_len"])
        return {"o": o.to(s["v"].dtype), "S": S}
    if case["op"] == "norm":
        return {"y": _plain_norm(case, s["x"], s["gate"], s["weight"], s["bias"], s["eps"]).to(s["y"].dtype)}
    names = ("q", "k", "v", "g", "beta", "S0") if case["op"] == "scan_backward" else ("x", "gate", "weight", "bias")
    leaves = {x: s[x].detach().requires_grad_() for x in names if s[x] is not None}
    a = {x: leaves.get(x) for x in names}
    if case["op"] == "scan_backward":
        o, S = _plain_scan(case, a["q"], a["k"], a["v"], a["g"], a["beta"], a["S0"], s["cu"], s["max_len"])
        outs, grads = [o], [s["do"].float()]
        if s["dS"] is not None:
            outs, grads = outs + [S], grads + [s["dS"]]
    else:
        outs, grads = [_plain_norm(case, a["x"], a["gate"], a["weight"], a["bias"], s["eps"])], [s["dy"].float()]
    got = torch.autograd.grad(outs, list(leaves.values()), grads)
    return {"d" + x: t for x, t in zip(leaves, got)}


def _workspace(s, backward):
    """The call's workspace, made once for a state, as a program that runs many steps keeps it."""
    if s["workspace"] is None:
        from sink_rank_recurrent_amd import sequence
        s["workspace"] = sequence.scan_workspace(s["case"]["rule"], s["q"], s["v"], s["case"]["n_seq"], backward=backward)
    return s["workspace"]


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "scan":
        o, S, _ = _steps(s)
        return {"o": o, "S": S}
    if case["op"] == "scan_backward":
        return _steps_back(s)
    return _norm64(s)


def _tokens64(s):
    """The inputs by position: a list of lengths in falling order makes the sequences still running a prefix."""
    cu = s["cu"].tolist()
    order = sorted(range(len(cu) - 1), key=lambda i: cu[i] - cu[i + 1])
    shared = s["case"]["heads"] // s["case"]["key_heads"]
    x = {name: None if s.get(name) is None else s[name].double() for name in ("q", "k", "v", "g", "beta", "do")}
    for name in ("q", "k"):
        x[name] = x[name].repeat_interleave(shared, 1)
    if x["g"].dim() == 2:
        x["g"] = x["g"][..., None]
    starts = torch.tensor([cu[i] for i in order], device="cuda")
    live = [cu[i + 1] - cu[i] for i in order]
    return x, order, starts, live


def _advance(rule, S, x, at):
    """One token of the running sequences: the decayed state, what is written, the new state."""
    kept = x["g"][at][..., None] * S
    k = x["k"][at][..., None]
    miss = x["v"][at] if rule == "mamba2" else x["v"][at] - (kept * k).sum(-2)
    u = miss if rule == "mamba2" else x["beta"][at][..., None] * miss
    return kept, miss, u, kept + k * u[..., None, :]


def _steps(s, every=0):
    """The recurrence as it is defined, a token of every sequence at a time; the states before each `every`-th token."""
    case = s["case"]
    x, order, starts, live = _tokens64(s)
    n, H, d_k, d_v = len(order), case["heads"], case["d_k"], case["d_v"]
    S = torch.zeros(n, H, d_k, d_v, device="cuda", dtype=torch.float64) if s["S0"] is None else s["S0"].double()[order]
    o = torch.zeros(case["tokens"], H, d_v, device="cuda", dtype=torch.float64)
    marks = []
    for t in range(live[0]):
        m = sum(length > t for length in live)
        if every and t % every == 0:
            marks.append(S[:m].clone())
        at = starts[:m] + t
        S[:m] = _advance(case["rule"], S[:m], x, at)[3]
        o[at] = (S[:m] * x["q"][at][..., None]).sum(-2)
    out = torch.empty_like(S)
    out[order] = S
    return o, out, marks


def _steps_back(s, every=16):
    """The gradients by the chain rule through each token, the states run again from every 16th one."""
    case = s["case"]
    rule, shared = case["rule"], case["heads"] // case["key_heads"]
    marks = _steps(s, every)[2]
    x, order, starts, live = _tokens64(s)
    n = len(order)
    dS = torch.zeros(n, case["heads"], case["d_k"], case["d_v"], device="cuda", dtype=torch.float64)
    if s["dS"] is not None:
        dS = s["dS"].double()[order]
    d = {name: torch.zeros_like(x[name]) for name in ("q", "k", "v", "g", "beta") if x[name] is not None}
    for block in reversed(range(len(marks))):
        S, steps = marks[block].clone(), []
        for t in range(block * every, min(live[0], (block + 1) * every)):
            m = sum(length > t for length in live)
            before = S[:m].clone()
            kept, miss, u, new = _advance(rule, before, x, starts[:m] + t)
            steps.append((t, m, before, kept, miss, u, new))
            S[:m] = new
        for t, m, before, kept, miss, u, new in reversed(steps):
            at = starts[:m] + t
            q, k, do = x["q"][at], x["k"][at], x["do"][at]
            d["q"][at] = (new * do[..., None, :]).sum(-1)
            dnew = dS[:m] + q[..., None] * do[..., None, :]
            du = (dnew * k[..., None]).sum(-2)
            dk = (dnew * u[..., None, :]).sum(-1)
            dkept = dnew
            if rule == "mamba2":
                d["v"][at] = du
            else:
                d["beta"][at] = (du * miss).sum(-1)
                dmiss = x["beta"][at][..., None] * du
                d["v"][at] = dmiss
                dk = dk - (kept * dmiss[..., None, :]).sum(-1)
                dkept = dnew - k[..., None] * dmiss[..., None, :]
            d["k"][at] = dk
            dg = (dkept * before).sum(-1)
            d["g"][at] = dg if rule == "kda" else dg.sum(-1, keepdim=True)
            dS[:m] = x["g"][at][..., None] * dkept
    out = {"d" + name: t for name, t in d.items()}
    for name in ("dq", "dk"):
        out[name] = out[name].unflatten(1, (case["key_heads"], shared)).sum(2)
    if rule != "kda":
        out["dg"] = out["dg"][..., 0]
    if s["S0"] is not None:
        out["dS0"] = torch.empty_like(dS)
        out["dS0"][order] = dS
    return out


def _norm64(s):
    case = s["case"]
    x, w = s["x"].double(), s["weight"].double()
    b = torch.zeros_like(w) if s["bias"] is None else s["bias"].double()
    z = None if s["gate"] is None else s["gate"].double()
    silu = case["activation"] == "silu"

    def act(t):
        sig = 1 / (1 + torch.exp(-t))
        return (t * sig, sig * (1 + t * (1 - sig))) if silu else (sig, sig * (1 - sig))

    h = x * act(z)[0] if case["gate"] == "before" else x
    mean = h.mean(-1, keepdim=True) if case["centered"] else 0.0
    rstd = 1 / torch.sqrt(((h - mean) ** 2).mean(-1, keepdim=True) + s["eps"])
    hat = (h - mean) * rstd
    n = hat * w + b
    if case["op"] == "norm":
        return {"y": n * act(z)[0] if case["gate"] == "after" else act(n)[0] if case["gate"] == "none" else n}
    dy = s["dy"].double()
    out = {}
    if case["gate"] == "after":
        dn, out["dgate"] = dy * act(z)[0], dy * n * act(z)[1]
    else:
        dn = dy * act(n)[1] if case["gate"] == "none" else dy
    over = (0, 1) if case["shared"] else (0,)
    out["dweight"] = (dn * hat).sum(over)
    if s["bias"] is not None:
        out["dbias"] = dn.sum(over)
    dhat = dn * w
    dh = dhat - hat * (dhat * hat).mean(-1, keepdim=True)
    if case["centered"]:
        dh = dh - dhat.mean(-1, keepdim=True)
    dh = dh * rstd
    if case["gate"] == "before":
        out["dgate"], dh = dh * x * act(z)[1], dh * act(z)[0]
    out["dx"] = dh
    return out
