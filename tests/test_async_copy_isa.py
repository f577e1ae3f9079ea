"""The asynchronous copy to LDS (async_copy in csrc/seed_scan.h) as machine
code, on the CPU: the compiler fills wait states in front of its own memory
instructions but does not look into an asm block.  A memory instruction may
read a scalar register five wait states after a vector instruction wrote it at
the earliest; sooner it takes the old value, here a copy from another address.
M0 has to be written one wait state before."""
import os
import re
import shutil
import subprocess

import pytest

from sink_rank_recurrent_amd import build

# bases the vector unit has only just made, one behind the other
SOURCE = """
#include "seed_scan.h"
__global__ void copies(const char* a, const uint32_t* at, uint32_t to, float* out) {
  __shared__ float lds[2048];
  const uint32_t x = at[threadIdx.x];
  seed::scan::async_copy(a + (size_t)x * 16, threadIdx.x * 16, to + x);
  seed::scan::async_copy(a + (size_t)x * 48, threadIdx.x * 16, to + x + 1024);
  seed::scan::async_wait();
  __syncthreads();
  out[threadIdx.x] = lds[threadIdx.x] + lds[threadIdx.x + 256];
}
"""


def _scalars(token):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", token)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", token)
    return {int(m[1])} if m else ({token} if token == "m0" else set())


def wait_states(text):
    """For each copy to LDS: wait states since a vector instruction wrote its
    base (None: not in its block), and since M0 was written."""
    found, block = [], []
    for raw in text.splitlines():
        line = raw.split(";")[0].strip()
        if re.match(r"[\w.$]+:", line):
            block = []
        if not line or line.startswith(".") or re.match(r"[\w.$]+:", line):
            continue
        op, _, rest = line.partition(" ")
        args = [x.strip() for x in rest.split(",")]
        if op.startswith("global_load_lds"):
            base, waited, since = _scalars(args[1].split()[0]), 0, {}
            for o, to in reversed(block):
                if o.startswith("v_") and _scalars(to) & base:
                    since.setdefault("base", waited)
                if to == "m0":
                    since.setdefault("m0", waited)
                waited += int(to, 0) + 1 if o == "s_nop" else 1
            found.append((since.get("base"), since.get("m0")))
        block.append((op, args[0]))
    return found


def test_the_count_itself():
    text = """f:
      v_readfirstlane_b32 s5, v1
      s_mov_b32 m0, s2
      s_nop 0
      global_load_lds_dwordx4 v0, s[4:5]
      s_nop 3
      global_load_lds_dwordx4 v0, s[6:7] offset:16"""
    assert wait_states(text) == [(2, 1), (None, 6)]


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="needs hipcc")
def test_base_and_m0_are_waited_for(tmp_path):
    source, out = tmp_path / "copies.hip", tmp_path / "copies.s"
    source.write_text(SOURCE)
    r = subprocess.run([build.hipcc(), *build.CXXFLAGS, "-I", build.CSRC, "--cuda-device-only", "-S",
                        str(source), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    copies = wait_states(out.read_text())
    assert len(copies) == 2 and all(base is not None for base, _ in copies), copies
    assert all(base >= 5 and m0 >= 1 for base, m0 in copies), copies
