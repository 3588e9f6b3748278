"""How the attention kernels wait, read from their sources (CPU).

A kernel that moves registers between its warpgroups (setmaxnreg) calls no
function: one compiled for the launch's registers may use more than the
caller's warps still hold."""
import os
import re

import pytest

from alibi_attention_block_gb300.build import CSRC


def code(file):
    with open(os.path.join(CSRC, file), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


KERNELS = sorted(f for f in os.listdir(CSRC) if f.startswith("attn") and f.endswith((".cu", ".cuh")))


@pytest.mark.parametrize("file", [f for f in KERNELS if "setmaxnreg" in code(f)])
def test_no_calls_where_registers_move(file):
    """The waits whose slow path is a call are mbar_wait and mbar_wait_slow."""
    assert re.findall(r"\bmbar_wait(?:_slow)?\(", code(file)) == []
