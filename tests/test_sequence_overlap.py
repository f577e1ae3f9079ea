"""Outputs and workspaces that lie over the offsets of a packed batch are
refused on the host, like those over any other input."""
import ctypes

import pytest

from test_sequence_abi import BACK, SCAN, SIZES, _call


def over(name):
    return lambda a: ctypes.c_void_p(a[name].value)


@pytest.mark.parametrize("name", ["o", "S", "ws"])
def test_scan_refuses_outputs_over_the_offsets(name):
    status, why = _call("seed_scan", SCAN, SIZES, {"cu": over(name)})
    assert status == 1 and "overlaps cu_seqlens" in why, why


@pytest.mark.parametrize("name", ["dq", "dk", "dv", "dg", "dbeta", "dS0", "ws"])
def test_backward_refuses_outputs_over_the_offsets(name):
    status, why = _call("seed_scan_backward", BACK, SIZES, {"cu": over(name)})
    assert status == 1 and "overlaps cu_seqlens" in why, why


def test_offsets_at_the_end_of_an_output():
    """n_seq + 1 offsets of 4 bytes: the last one counts."""
    values = SIZES["tokens"] * SIZES["heads"] * SIZES["d_v"] * 2
    last = {"cu": lambda a: ctypes.c_void_p(a["o"].value - 4 * SIZES["n_seq"])}
    assert _call("seed_scan", SCAN, SIZES, last)[0] == 1
    last = {"cu": lambda a: ctypes.c_void_p(a["o"].value + values - 4)}
    assert _call("seed_scan", SCAN, SIZES, last)[0] == 1
