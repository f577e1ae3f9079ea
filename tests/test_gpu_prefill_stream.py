"""Memory of what prefill returns, when it runs on a stream of its own."""
import pytest
import torch

from gpu_util import requires_gpu
from sink_rank_recurrent_amd import binding
from test_gpu_scan import inputs

pytestmark = [pytest.mark.gpu, requires_gpu]


def test_states_freed_while_the_caller_still_reads_them():
    """The dense states come from the given stream's pool, and the caller
    reads them on its own stream.  Let go of there, the memory may not go to
    the next allocation on the given stream before those reads are done."""
    H, d = 2, 128
    x = inputs("gdn", 200, H, H, d, d, 2, torch.bfloat16, 51, initial=False)
    o = torch.empty_like(x["v"])
    cu = torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda")
    st = binding.ShallowState("gdn", 2, H, d, d, 16, 16, torch.ones(H, d, device="cuda"))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    S = st.prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], o, cu_seqlens=cu, stream=side)
    torch.cuda.synchronize()
    want, at, shape = S.cpu(), S.data_ptr(), S.shape
    torch.cuda._sleep(200_000_000)      # the caller's stream is busy ...
    got = S.clone()                     # ... and reads behind that
    del S
    with torch.cuda.stream(side):
        other = [torch.zeros(shape, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != at for t in other)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), want)
