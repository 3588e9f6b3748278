"""More refusals of the paged cache's calls and of the rotary's plan, without a GPU: outputs that lie
on top of themselves, spans; and where a paged decode step takes one launch."""
import pytest

import alibi_attention_block_gb300 as blk
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


@pytest.mark.parametrize("kind,H,Hk,d,most", [  # units (eight query heads of a kv head) of one launch
    (1, 16, 16, 64, 1024), (1, 64, 16, 64, 1024), (1, 32, 4, 64, 512), (0, 16, 16, 64, 512), (1, 32, 8, 128, 512),
    (0, 16, 4, 128, 512), (0, 16, 1, 128, 256), (1, 32, 2, 160, 256), (0, 32, 8, 160, 256)])
def test_few_units_take_one_launch(lib, kind, H, Hk, d, most):  # noqa: F811
    """Many sequences of few keys take two launches, and need a workspace for them."""
    def need(batch, keys):
        fields = (9, 16, Hk, d, batch, keys // 16, Hk * 16 * d, kind)
        return blk.attn_decode_paged_workspace_size(blk.decode_paged_desc(fields, H, H * d, d))
    assert need(most // Hk, 512) == 0 and need(1, 16) == 0
    assert need(most // Hk + 1, 512) > 0 and need(most // Hk + 1, 16) > 0 and need(1, 528) > 0


@pytest.mark.parametrize("span", [2 ** 32 + 64, 2 ** 31, -2 ** 32 + 64, 64.5, float("nan"), float("inf")])
def test_spans_that_are_no_32_bit_numbers(lib, span):  # noqa: F811
    """... were cut to the 32 bits, or to the whole number, that the library took for a span."""
    with pytest.raises(ValueError):
        blk.rope_plan(span)
    assert blk.rope_plan(64.0) is blk.rope_plan(64)
