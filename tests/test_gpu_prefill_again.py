"""A state that has run takes new prompts: prefill leaves it as it leaves a
new one, whatever steps, windows and compressions there were before."""
import pytest
import torch

from gpu_util import requires_gpu
from sink_rank_recurrent_amd import binding, sequence
from test_gpu_scan import inputs

pytestmark = [pytest.mark.gpu, requires_gpu]

B, H, R, W = 3, 2, 16, 16


def args(x):
    return x["q"], x["k"], x["v"], x["g"], x["beta"]


def steps(st, rule, dims, n, seed):
    outs = []
    for t in range(n):
        x = inputs(rule, B, H, H, *dims, B, torch.bfloat16, seed + t, initial=False)
        o = torch.empty(B, H, dims[1], device="cuda")
        if isinstance(st, binding.ScheduledState):
            st.step(*args(x), o)
        else:
            st.step_and_maybe_compress(*args(x), o)
        outs.append(o)
    return outs


@pytest.mark.parametrize("rule,dims", [("gdn", (128, 128)), ("kda", (64, 64)), ("mamba2", (128, 64))])
@pytest.mark.parametrize("form", ["fp32", "lazy", "h16", "scheduled", "scheduled 6", "scheduled 6 aside"])
@pytest.mark.parametrize("before", [5, W + 3, 2 * W + 9])
def test_prefill_of_a_used_state_is_that_of_a_new_one(rule, dims, form, before):
    vbar = torch.randn(H, dims[1], device="cuda", generator=torch.Generator("cuda").manual_seed(4))

    def make():
        if form == "h16":
            return binding.ShallowState16(rule, B, H, *dims, R, W, vbar)
        if form.startswith("scheduled"):
            return binding.ScheduledState(rule, B, H, *dims, R, W, 6 if "6" in form else 0, vbar, [0, 4, 9],
                                          side_streams=2 if "aside" in form else 0)
        return binding.ShallowState(rule, B, H, *dims, R, W, vbar, lazy=form == "lazy")

    T = 90
    x = inputs(rule, B * T, H, H, *dims, B, torch.bfloat16, 31, initial=False)
    cu = torch.tensor([0, 40, 41, B * T], dtype=torch.int32, device="cuda")
    o = torch.empty_like(x["v"])
    new, used = make(), make()
    S = new.prefill(*args(x), o, cu_seqlens=cu)
    other = inputs(rule, B * T, H, H, *dims, B, torch.bfloat16, 32, initial=False)
    used.prefill(*args(other), o, cu_seqlens=cu)
    steps(used, rule, dims, before, 100)
    assert torch.equal(used.prefill(*args(x), o, cu_seqlens=cu), S)
    if form.startswith("scheduled"):
        assert used.t == 0 and not used.pending
    else:
        assert (used.r, used.limit) == (new.r, new.limit)
    n = 2 * W + 9
    for t, (a, b) in enumerate(zip(steps(new, rule, dims, n, 200), steps(used, rule, dims, n, 200))):
        assert torch.equal(a, b), t
