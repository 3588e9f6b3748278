"""blk_attn_prefill_packed where a CTA takes several work items, and its ALiBi
kernels at head_dim 128 and 160, against the fp64 oracle (GPU).

With more items than CTAs an item's last product and read-out run beside the
next item's first tiles, rings and barrier phases go on across items, and
items with and without a second query tile follow one another. What such a
call gives each prompt has to be, bit for bit, what the prompt gets by itself
(a call of a few items, none of them a CTA's second), and within the oracle's
bound. That bound, and the roundings it is derived from, are those of
test_gpu_packed.py.
"""
import numpy as np
import pytest
import torch

import alibi_attention_block_gb300 as blk
import oracle
from tests.parity import to_dev
from tests.test_gpu_packed import check_rows, ends, inputs, reference, slopes_of, table

pytestmark = pytest.mark.gpu

CTAS = 152  # at most: one per SM


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def positions_per_unit(H, Hk, d, alibi):
    """Of a work item: a pair of query tiles, or one where a slope per row is
    needed (ALiBi over grouped heads above head_dim 64)."""
    if d == 64:
        return 256
    G = H // Hk
    R = 128 // min(G, 16) // 8 * 8
    return R if alibi and G > 1 else 2 * R


def items(H, Hk, d, alibi, lens):
    unit = positions_per_unit(H, Hk, d, alibi)
    per_unit = H if d == 64 else Hk * -(-(H // Hk) // 16)
    return sum(-(-n // unit) for n in lens) * per_unit


# odd and even numbers of query tiles, with a full and a part-filled last one
MIXED = [1, 257, 128, 64, 513, 129, 0, 256, 385, 2, 127, 130, 400, 63, 65, 640]

ROUNDS = [
    # H, Hk, d, lens, prefix, alibi, dtype
    (24, 24, 64, MIXED, 0, False, "fp16"),
    (24, 8, 64, MIXED, 200, False, "bf16"),
    (24, 24, 64, MIXED, 128, True, "bf16"),
    (24, 24, 128, MIXED, 0, False, "bf16"),
    (24, 24, 128, MIXED, 131, False, "fp16"),
    (24, 24, 128, MIXED, 0, True, "fp16"),
    (24, 24, 128, MIXED, 260, True, "bf16"),
    (32, 8, 128, MIXED, 0, False, "bf16"),
    (36, 12, 128, MIXED, 77, False, "fp16"),       # 40 positions a tile
    (32, 8, 128, MIXED, 0, True, "bf16"),
    (36, 12, 128, MIXED, 129, True, "fp16"),
    (24, 24, 160, MIXED, 0, False, "fp16"),
    (24, 24, 160, MIXED, 70, False, "bf16"),
    (24, 24, 160, MIXED, 0, True, "bf16"),
    (24, 24, 160, MIXED, 193, True, "fp16"),
    (32, 8, 160, MIXED, 0, False, "fp16"),
    (36, 12, 160, MIXED, 77, False, "bf16"),
    (32, 8, 160, MIXED, 0, True, "fp16"),
    (44, 2, 160, MIXED, 129, True, "bf16"),        # 16 + 6 heads a group
    (32, 8, 160, MIXED, 64, True, "bf16"),
]


def name_of(c):
    return "H{}Hk{}d{}n{}P{}{}_{}".format(c[0], c[1], c[2], len(c[3]), c[4], "_alibi" if c[5] else "", c[6])


@pytest.mark.parametrize("case", ROUNDS, ids=name_of)
def test_rounds_of_items(case):
    H, Hk, d, lens, P, alibi, dt = case
    assert items(H, Hk, d, alibi, lens) > 3 * CTAS
    cu = ends(lens)
    q, k, v, kp, vp = inputs(H, Hk, cu[-1], d, P, dt, 300 + H + d + P)
    ref_slopes, dev_slopes = slopes_of(H, alibi)
    args = dict(k_prefix=to_dev(kp), v_prefix=to_dev(vp), alibi=alibi, slopes=dev_slopes)
    qd, kd, vd = to_dev(q), to_dev(k), to_dev(v)
    o = blk.attn_prefill_packed(qd, kd, vd, table(cu), **args)
    blk.check_device_status()
    assert torch.equal(o, blk.attn_prefill_packed(qd, kd, vd, table(cu), **args))
    # the same units in another order, and so on other CTAs: the list in the workspace
    assert torch.equal(o, blk.attn_prefill_packed(qd, kd, vd, table(cu + [cu[-1]] * 300), **args))
    for i, n in enumerate(lens):
        if n == 0:
            continue
        a, b = cu[i], cu[i + 1]
        alone = [t[:, a:b].contiguous() for t in (qd, kd, vd)]
        got = blk.attn_prefill_packed(*alone, table([0, n]), **args)
        assert torch.equal(o[a:b], got), f"{case} prompt {i}: not what it gets by itself"
    for i in (0, 1, 5, 8, 15):
        check_rows(o[cu[i]:cu[i + 1]], reference(q, k, v, cu[i], lens[i], kp, vp, ref_slopes), dt,
                   f"{case} prompt {i}")


LENS = [1, 0, 63, 64, 65, 2, 127, 128, 129, 255, 256, 257, 0, 33, 520]
ALIBI = [
    # a kv head per query head at head_dim 160, whose rows' first key tiles (64
    # keys, from the diagonal down) may hold nothing that they see
    (2, 2, 160, LENS, 0, "bf16"),
    (2, 2, 160, LENS, 0, "fp16"),
    (4, 4, 160, LENS, 64, "fp16"),
    (2, 2, 160, LENS, 100, "bf16"),
    (3, 3, 160, LENS, 257, "bf16"),     # given slopes
    (3, 3, 160, [300, 1, 128], 1, "fp16"),
    (1, 1, 160, [1], 0, "bf16"),
    (5, 5, 160, [640, 639, 641], 0, "fp16"),
    # and the neighbouring forms
    (2, 2, 128, LENS, 0, "bf16"),
    (3, 3, 128, LENS, 100, "fp16"),
    (8, 2, 128, LENS, 0, "fp16"),
    (6, 2, 128, LENS, 100, "bf16"),     # blocks of 40 positions across key tiles
    (8, 2, 160, LENS, 100, "bf16"),
    (5, 1, 160, LENS, 0, "fp16"),       # blocks of 24 positions
]


@pytest.mark.parametrize("case", ALIBI, ids=lambda c: name_of(c[:5] + (True,) + c[5:]))
def test_alibi_matches_oracle(case):
    H, Hk, d, lens, P, dt = case
    front, back = 5, 150  # rows of no prompt, poisoned
    cu = ends(lens, front)
    T = cu[-1] + back
    q, k, v, kp, vp = inputs(H, Hk, T, d, P, dt, 700 + H + d + P)
    qd, kd, vd = to_dev(q), to_dev(k), to_dev(v)
    for t in (qd, kd, vd):
        t[:, :front] = float("inf")
        t[:, cu[-1]:] = float("nan")
    out = torch.full((T, H, d), 7.0, dtype=qd.dtype, device="cuda")
    ref_slopes, dev_slopes = slopes_of(H, True)
    blk.attn_prefill_packed(qd, kd, vd, table(cu), k_prefix=to_dev(kp), v_prefix=to_dev(vp), alibi=True,
                            slopes=dev_slopes, out=out)
    blk.check_device_status()
    for i, n in enumerate(lens):
        if n:
            check_rows(out[cu[i]:cu[i + 1]], reference(q, k, v, cu[i], n, kp, vp, ref_slopes), dt,
                       f"{case} prompt {i}")
    assert (out[:front] == 7).all() and (out[cu[-1]:] == 7).all()


SHAPES = [(2, 2, 64), (2, 2, 128), (8, 2, 128), (6, 2, 128), (2, 2, 160), (8, 2, 160), (5, 1, 160)]


@pytest.mark.parametrize("H,Hk,d", SHAPES)
def test_alibi_prompts_do_not_touch_each_other(H, Hk, d):
    """A prompt full of NaN and infinities leaves the others' bits alone."""
    lens = [100, 57, 300, 1, 70]
    cu = ends(lens)
    q, k, v, kp, vp = inputs(H, Hk, cu[-1], d, 150, "bf16", 5)
    qd, kd, vd = to_dev(q), to_dev(k), to_dev(v)
    args = dict(k_prefix=to_dev(kp), v_prefix=to_dev(vp), alibi=True, slopes=slopes_of(H, True)[1])
    good = blk.attn_prefill_packed(qd, kd, vd, table(cu), **args)
    for i in (1, 3):
        for t, bad in ((qd, float("nan")), (kd, float("inf")), (vd, float("nan"))):
            t[:, cu[i]:cu[i + 1]] = bad
    o = blk.attn_prefill_packed(qd, kd, vd, table(cu), **args)
    blk.check_device_status()
    for i in (0, 2, 4):
        assert torch.equal(o[cu[i]:cu[i + 1]], good[cu[i]:cu[i + 1]])


@pytest.mark.parametrize("H,Hk,d", SHAPES)
def test_alibi_list_in_the_workspace(H, Hk, d):
    lens = [100, 257, 300, 1, 513]
    cu = ends(lens)
    q, k, v, kp, vp = inputs(H, Hk, cu[-1], d, 150, "fp16", 17)
    args = to_dev(q), to_dev(k), to_dev(v)
    more = dict(k_prefix=to_dev(kp), v_prefix=to_dev(vp), alibi=True, slopes=slopes_of(H, True)[1])
    a = blk.attn_prefill_packed(*args, table(cu), **more)
    b = blk.attn_prefill_packed(*args, table(cu + [cu[-1]] * 300), **more)
    blk.check_device_status()
    assert torch.equal(a, b)


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("H,Hk,d", SHAPES)
def test_alibi_scores_that_move_the_maximum(H, Hk, d, rising):
    """Scores that fall along the prompt by more than a weak slope's bias rises:
    walked down from the diagonal, the running maximum moves at every tile.
    (Scores times log2(e) stay below 2^6, biases too, so an exponent's sums stay
    below 2^7: each of their roundings, at most 2^-18, is a sixteenth of what the
    bound allows them.)"""
    n, P = 500, 200
    q, k, v, kp, vp = inputs(H, Hk, n, d, P, "bf16", 8)
    ramp = torch.linspace(0.0, 3.0, P + n) if rising else torch.linspace(3.0, 0.0, P + n)
    q = torch.ones_like(q)
    k = (ramp[P:, None] * torch.ones(Hk, n, d)).to(torch.bfloat16)
    kp = (ramp[:P, None] * torch.ones(Hk, P, d)).to(torch.bfloat16)
    s = np.linspace(0.004, 0.05, H).astype(np.float32)
    o = blk.attn_prefill_packed(to_dev(q), to_dev(k), to_dev(v), table([0, n]), k_prefix=to_dev(kp),
                                v_prefix=to_dev(vp), alibi=True, slopes=torch.from_numpy(s).cuda())
    blk.check_device_status()
    check_rows(o, reference(q, k, v, 0, n, kp, vp, s.astype(np.float64)), "bf16", f"{H}/{Hk} x {d}")


@pytest.mark.parametrize("H,Hk,d", SHAPES)
def test_alibi_graph_replay(H, Hk, d):
    """A captured call follows new tables and inputs."""
    q, k, v, kp, vp = inputs(H, Hk, 600, d, 140, "bf16", 12)
    qd, kd, vd, kpd, vpd = map(to_dev, (q, k, v, kp, vp))
    cu = table([0, 250, 251, 600])
    slopes = slopes_of(H, True)[1]

    def call(**kw):
        return blk.attn_prefill_packed(qd, kd, vd, cu, k_prefix=kpd, v_prefix=vpd, alibi=True, slopes=slopes, **kw)

    out = torch.zeros((600, H, d), dtype=torch.bfloat16, device="cuda")
    call(out=out)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(out=out)
    for tab in ([0, 250, 251, 600], [0, 10, 400, 600], [0, 600, 600, 600]):
        cu.copy_(table(tab))
        qd.copy_(qd.flip(1))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, call())
        blk.check_device_status()
    refs, _ = slopes_of(H, True)
    check_rows(got, reference(qd.cpu(), k, v, 0, 600, kp, vp, refs), "bf16", f"{H}/{Hk} x {d}")


def test_scales_changed_in_place():
    """A 0-dim tensor given as scale is read at each call (both entry points)."""
    q, k, v, _, _ = inputs(2, 2, 100, 64, 0, "bf16", 21)
    args = to_dev(q), to_dev(k), to_dev(v), table([0, 100])
    step = (to_dev(q)[:, :3].transpose(0, 1).contiguous(), None, None,
            to_dev(k).view(1, 2, 100, 64).repeat(3, 1, 1, 1), to_dev(v).view(1, 2, 100, 64).repeat(3, 1, 1, 1),
            torch.tensor([100, 7, 33], dtype=torch.int32, device="cuda"))
    for device in ("cpu", "cuda"):
        t = torch.tensor(0.25, device=device)
        for value in (0.25, 0.5):
            t.fill_(value)
            assert torch.equal(blk.attn_prefill_packed(*args, scale=t), blk.attn_prefill_packed(*args, scale=value))
            assert torch.equal(blk.attn_decode_shared(*step, scale=t), blk.attn_decode_shared(*step, scale=value))
    ref = reference(q, k, v, 0, 100, scale=0.5)
    check_rows(blk.attn_prefill_packed(*args, scale=t), ref, "bf16", "scale 0.5")


@pytest.mark.parametrize("H,Hk,d,n", [(4, 1, 64, 13200), (2, 2, 128, 16500), (2, 2, 160, 14000)])
def test_a_long_idle_second_tile(H, Hk, d, n):
    """Prompts of one token behind a prefix of 2^20, and one prompt of two query
    tiles behind them: the second tile's softmax warps have nothing to do for
    2.6 to 3 seconds, longer than a wait that has lost its arrival may last, and
    then their part of the last prompt. It gets what it gets by itself."""
    P, last = 1 << 20, 250
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    q, k, v, kp, vp = (torch.randn(s, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
                       for s in ((H, n + last, d), (Hk, n + last, d), (Hk, n + last, d), (Hk, P, d), (Hk, P, d)))
    pre = dict(k_prefix=kp, v_prefix=vp)
    o = blk.attn_prefill_packed(q, k, v, table(list(range(n + 1)) + [n + last]), **pre)
    blk.check_device_status()
    alone = [t[:, n:].contiguous() for t in (q, k, v)]
    assert torch.equal(o[n:], blk.attn_prefill_packed(*alone, table([0, last]), **pre))
    first = [t[:, :100].contiguous() for t in (q, k, v)]
    assert torch.equal(o[:100], blk.attn_prefill_packed(*first, table(list(range(101))), **pre))
    blk.check_device_status()
