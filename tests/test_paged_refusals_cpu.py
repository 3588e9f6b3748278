"""More refusals of the paged cache's calls and of the rotary's plan, without a GPU: outputs that lie
on top of themselves."""
import pytest

from tests.test_paged_abi_cpu import EINVAL, FAKE, append, lib, rope  # noqa: F401

OVERLAPS = [  # strides of heads and tokens of an output [4, 10, 128]
    (0, 128), (1280, 0), (0, 0), (128, 128), (64, 512), (1272, 128), (1280, 120), (128, 504), (640, 128)]
APART = [(1280, 128), (128, 512), (1 << 40, 136), (136, 536), (128, 1 << 40)]


@pytest.mark.parametrize("head,token", OVERLAPS)
def test_outputs_that_overlap_themselves(lib, head, token):  # noqa: F811
    """Written by several threads at once, in no order."""
    out = {"q_out_head_stride": head, "q_out_token_stride": token}
    assert rope(lib, **out) == EINVAL
    assert rope(lib, n_k_heads=4, k_out_head_stride=head, k_out_token_stride=token) == EINVAL
    same = {**out, "q_head_stride": head, "q_token_stride": token}  # in place, too
    assert rope(lib, qo=FAKE, **same) == EINVAL
    assert append(lib, n_heads=4, q=FAKE, qo=2 * FAKE, **out) == EINVAL
    assert append(lib, n_heads=4, q=FAKE, qo=FAKE, **same) == EINVAL


@pytest.mark.parametrize("head,token", APART)
def test_outputs_apart_are_not_refused(lib, head, token):  # noqa: F811
    """... for that: what the calls say is the next thing that is wrong with them."""
    out = {"q_out_head_stride": head, "q_out_token_stride": token, "q_head_stride": 2 * 1280}
    one = {"q_out_head_stride": 0, "q_out_token_stride": 0, "q_token_stride": 256, "n_heads": 1}
    assert rope(lib, qo=FAKE, **out) == EINVAL and b"in place" in lib.blk_last_error()
    assert rope(lib, qo=FAKE, tokens=1, **one) == EINVAL and b"in place" in lib.blk_last_error()
    assert append(lib, n_heads=4, q=FAKE, qo=FAKE, **out) == EINVAL and b"in place" in lib.blk_last_error()
