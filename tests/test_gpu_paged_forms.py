"""The paged decode step's two forms, on both sides of the rule that chooses (few keys and few
units: one launch without a workspace), against the definition in 64 bits."""
import pytest

import alibi_attention_block_gb300 as blk
from tests.test_gpu_paged import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


@pytest.mark.parametrize("B,H,Hk,d,page,bits,most", [
    (64, 16, 8, 128, 32, 8, 512), (65, 16, 8, 128, 32, 8, 512), (256, 4, 4, 64, 64, 8, 1024), (257, 4, 4, 64, 64, 8, 1024),
    (128, 8, 2, 160, 16, 16, 256), (129, 8, 2, 160, 16, 16, 256), (171, 48, 3, 64, 16, 16, 512), (86, 48, 3, 128, 16, 16, 512),
    (85, 48, 3, 128, 16, 16, 512), (129, 32, 4, 64, 16, 8, 512)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_both_sides_of_the_rule(B, H, Hk, d, page, bits, most, dt):
    lens = [(37 * i) % 190 for i in range(B)]
    lens[1] = 512
    cols = 512 // page
    size = blk.attn_decode_paged_workspace_size(blk.decode_paged_desc(
        (9, page, Hk, d, B, cols, Hk * page * d, 1 if bits == 8 else 0), H, H * d, d))
    units = B * Hk * ((H // Hk + 7) // 8)
    assert (size == 0) == (units <= most)
    run(B, H, Hk, d, page, lens, dt, bits, False, seed=B, room=0)
