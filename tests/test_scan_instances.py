"""The kernels in the built library that go from chunk to chunk: every one is
reached by some call."""
import os
import re

import pytest

from sink_rank_recurrent_amd import binding

NAME = re.compile(rb"(chain|wide)_(forward|reverse)_kernelILi(\d)ELi(\d+)ELi(\d)E([tf]?)L([ib])(\d)EE")


@pytest.mark.skipif(not os.path.exists(binding.LIB_PATH), reason="needs the built library")
def test_segments_are_walked_by_four_waves():
    """Where a sequence goes in segments a workgroup has four waves, so what a
    segment carries (forward mode 2) or passes back (reverse, local) has no
    eight-wave form."""
    found = set(NAME.findall(open(binding.LIB_PATH, "rb").read()))
    assert found
    for file, way, rule, d_k, waves, _, _, mode in found:
        carries = mode == (b"2" if way == b"forward" else b"1")
        assert waves == b"4" or not carries, (file, way, rule, d_k, waves, mode)
    assert any(waves == b"8" for _, _, _, _, waves, _, _, _ in found)
