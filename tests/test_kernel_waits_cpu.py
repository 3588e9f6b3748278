"""How the attention kernels wait, read from their sources (CPU).

A kernel that moves registers between its warpgroups (setmaxnreg) calls no
function: one compiled for the launch's registers may use more than the
caller's warps still hold.

A block whose wait gave up ends, and its shared memory and TMEM go to the next
one: whatever its other warps met, the loading thread first waits for the copies
it has in flight, each issuing thread for its products."""
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


def loading_threads(text):
    """Of each loading thread: the barriers its copies complete, and the code
    from its last copy to the products that follow it."""
    names, last = set(), None
    for m in re.finditer(r"mbar_expect_tx\((?:bar\.)?(\w+)|tma_load_\w+\(|tc_mma_\w+\(", text):
        if m.group(1):
            names.add(m.group(1))
        elif m.group(0).startswith("tma"):
            last = m.end()
        elif last is not None:
            yield names, text[last:m.start()]
            names, last = set(), None


@pytest.mark.parametrize("file", [f for f in KERNELS if "tc_mma_" in code(f)])
def test_a_block_ends_behind_its_copies_and_products(file):
    text = code(file)
    threads = list(loading_threads(text))
    assert threads
    for names, ending in threads:
        assert names
        # (one loop over the barriers of K and then V, which lie together)
        both = re.search(r"i < 2 \* kStages[^;]*;[^}]*mbar_wait\w*\([^;]*k_full\(0\) \+ 8u \* i\b", ending, re.S)
        for name in sorted(names):
            assert re.search(r"mbar_wait\w*\([^;]*\b%s\(" % name, ending) or both and name == "v_full", \
                f"copies of {name} are not waited for"
    # each place of issuing threads commits its products to a barrier that is waited for
    for call in (r"tc_commit\((?:bar\.)?drain[^;]*\);", r"mbar_wait\w*\((?:bar\.)?drain[^;]*, 0, a\.err\);"):
        assert len(re.findall(call, text)) == len(threads)
