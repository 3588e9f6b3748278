"""How exact the turn itself is (blk_rope_positions, and the keys and queries of blk_kv_append_paged):
pairs (x, y) for which x cos a - y sin a nearly vanishes, so that the output's rounding, relative to the value, hides
nothing.

Error, in parts of |x| + |y| (2^-24: half a step of 32 bits, relative): the angle's 32 bits of a turn are 2^-30
of a radian off; its float, the constant and their product 3 2^-24 of an eighth of a turn, 2.36 2^-24; the cosine's series
2.5e-8 = 0.42 2^-24, its roundings 1.4 2^-24, its slope 0.71: 3.5 2^-24; the sine's series and roundings 0.85 2^-24, its angle's
part 1.7 2^-24 and the product's rounding 2^-24: 3.5 2^-24. Both below 2^-22. The hardware's sine and cosine
(2^-21.4 at best) are not."""
import numpy as np
import pytest
import torch

import alibi_attention_block_gb300 as blk
from tests import paged_ref as ref
from tests.parity import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def pairs(angle, rng):
    """x, y with x cos a - y sin a as near to 0 as eleven bits allow, of about 1000."""
    c, s = np.cos(angle)[..., None], np.sin(angle)[..., None]
    n = rng.integers(1024, 2048, angle.shape + (256,)).astype(np.float64)
    swap = np.abs(c) > np.abs(s)  # the larger factor's number is the one that is rounded
    x = np.where(swap, np.round(n * s / np.where(swap, c, 1)), n)
    y = np.where(swap, n, np.round(n * c / np.where(swap, 1, s)))
    best = np.abs(x * c - y * s).argmin(-1)[..., None]
    return np.take_along_axis(x, best, -1)[..., 0], np.take_along_axis(y, best, -1)[..., 0]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("span,d", [(128, 128), (40, 160), (30, 32)])
@pytest.mark.parametrize("far", [300, 1 << 20])
def test_turn(far, span, d, interleaved):
    rng = np.random.default_rng(span + far)
    T = 2000
    pos = rng.integers(0, far, T)
    th = ref.thetas(span)
    x, y = pairs(pos[:, None] * th, rng)  # [T, pairs]
    row = np.zeros((1, T, d))
    if interleaved:
        row[0, :, 0:span:2], row[0, :, 1:span:2] = x, y
    else:
        row[0, :, :span // 2], row[0, :, span // 2:span] = x, y
    q = torch.tensor(row, device="cuda").half()
    assert np.array_equal(f64(q.float()), row)
    plan = blk.rope_plan(span, 10000.0, interleaved=interleaved)
    positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
    want, mag = ref.turn(row, pos, th, interleaved)
    bound = 2.0 ** -22 * mag + 2.0 ** -11 * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -25
    a = blk.rope_positions(q, positions, plan)
    err = np.abs(f64(a.float()) - want)
    assert (err <= bound).all(), f"{float((err / bound).max()):.2f} of the bound"
    # the append's: keys by the angles' table, queries by their own, at given positions
    page = 128
    cache = [torch.zeros((T // page + 1, 1, page, d), dtype=torch.float16, device="cuda") for _ in "kv"]
    table = torch.arange(T // page + 1, dtype=torch.int32, device="cuda")[None]
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    b = blk.kv_append_paged(q, q, *cache, table, n, cu_seqlens=torch.tensor([0, T], dtype=torch.int32, device="cuda"), rope=plan,
                            positions=positions, q=q)
    assert torch.equal(a, b)
    assert torch.equal(a[0], cache[0].transpose(0, 1).flatten(1, 2)[0, :T])
