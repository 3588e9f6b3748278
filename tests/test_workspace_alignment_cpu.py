"""Workspace sizes against the alignment that their kernels store with (CPU)."""
import ctypes as C
import os
import re

import pytest

from alibi_attention_block_gb300 import _abi, build


@pytest.mark.parametrize("desc", [
    (40, 200, 16, 2, 64, 700, -1.0, 0), (5, 300, 8, 8, 128, 1000, -1.0, 0), (6, 900, 8, 4, 128, 0, -1.0, 1)])
def test_room_for_the_first_boundary(desc):
    """blk_attn_decode_shared's kernel stores 32 bytes at a time and its
    workspace may be aligned to 16: beside its parts, of whole 256 bytes each, it
    has room for the step to the first boundary of 32."""
    with open(os.path.join(build.CSRC, "attn_shared.cuh"), encoding="utf-8") as f:
        assert re.search(r"st\.global\.v8\.f32", f.read())
    build.build()
    need = C.c_size_t(0)
    d = _abi.DecodeSharedDesc(*desc)
    assert _abi.load().blk_attn_decode_shared_workspace_size(C.byref(d), C.byref(need)) == _abi.BLK_OK
    assert need.value % 256 == 32 - 16
