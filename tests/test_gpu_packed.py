"""GPU parity of blk_attn_prefill_packed (causal attention over packed prompts
of different lengths, optionally behind a shared prefix) against the fp64
oracle, prompt by prompt, through the C ABI.

Error bound of one output element (u = eps / 2 of the storage type, half a
step): each weight p is rounded once to the storage type (relative error u;
fp16 weights below its smallest normal, at most 2^-25 absolute against a
largest weight of at least 1), the output once more (u |o|). Scores,
exponentials and sums are fp32: with |score| log2(e) <= 2^6 in these cases
they add less than 2^-14 relative (the exponent's rounding 2^-18 ln 2, ex2's
2^-22, a tile's accumulation). So
    |err| <= (u + 2^-14) sum_j p_j |v_j| + u |o| + n 2^-25 max |v|.
"""
import dataclasses

import numpy as np
import pytest
import torch

import alibi_attention_block_gb300 as blk
import oracle
import workloads
from tests.parity import ABS_TOL, check, f64, to_dev
from tests.test_storage_budget import POST_NORM_ABS_TOL
from workloads import BLOCK_CONFIGS, draw, scaled

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def reference(q, k, v, start, n, kp=None, vp=None, slopes=None, scale=None):
    """fp64 (o [n, H, d], sum p|v|) of the prompt at rows start .. start+n-1."""
    q, k, v = (f64(t)[None, :, start:start + n] for t in (q, k, v))
    P = 0
    if kp is not None:
        P = kp.shape[1]
        k = np.concatenate([f64(kp)[None], k], axis=2)
        v = np.concatenate([f64(vp)[None], v], axis=2)
    pos = np.arange(P, P + n)
    o, a = (oracle.attention(q, k, w, scale=scale, slopes=slopes, q_positions=pos)[0].transpose(1, 0, 2)
            for w in (v, np.abs(v)))
    return o, a, P + n, float(np.abs(v).max())


def check_rows(got, ref, dt, name):
    o, a, keys, vmax = ref
    u = HALF_STEP[dt]
    bound = (u + 2.0 ** -14) * a + u * np.abs(o) + keys * 2.0 ** -25 * vmax
    err = np.abs(f64(got) - o)
    assert np.isfinite(f64(got)).all(), f"{name}: non-finite output"
    assert (err <= bound).all(), f"{name}: error {err.max():.3e}, {float((err / bound).max()):.2f} of the bound"


def inputs(H, Hk, T, d, P, dt, seed):
    q, k, v = draw((H, T, d), dt, seed), draw((Hk, T, d), dt, seed + 1), draw((Hk, T, d), dt, seed + 2)
    kp = draw((Hk, P, d), dt, seed + 3) if P else None
    vp = draw((Hk, P, d), dt, seed + 4) if P else None
    return q, k, v, kp, vp


def ends(lens, first=0):
    return [first + int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


def table(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


LENS = [1, 0, 127, 128, 129, 2, 255, 256, 257, 0, 33, 520]
CASES = [
    # H, Hk, d, lens, prefix, alibi, dtype
    (4, 4, 64, LENS, 0, False, "bf16"),
    (4, 2, 64, LENS, 0, True, "fp16"),
    (2, 2, 64, [1], 0, False, "fp16"),
    (2, 1, 64, [0, 0, 1, 1, 1, 0], 0, True, "bf16"),
    (2, 2, 64, [700, 3, 65], 1, False, "bf16"),
    (2, 2, 64, [300, 1, 128], 128, True, "fp16"),
    (4, 1, 64, [40, 513, 7], 333, True, "bf16"),
    (2, 2, 128, LENS, 0, False, "bf16"),
    (2, 2, 128, [300, 1, 128], 257, True, "fp16"),
    (8, 2, 128, LENS, 0, False, "fp16"),
    (8, 2, 128, LENS, 200, True, "bf16"),
    (3, 1, 128, [45, 300, 0, 81], 5, False, "bf16"),      # 40 positions a unit
    (6, 2, 128, [130, 41, 40, 39], 0, False, "fp16"),
    (32, 1, 128, [17, 70], 130, False, "bf16"),           # two head chunks a group
    (8, 2, 160, LENS, 0, False, "bf16"),
    (4, 1, 160, [200, 129, 1, 0, 64], 129, True, "fp16"),
    (2, 2, 160, [1, 260], 0, False, "fp16"),
    (3, 1, 128, [45, 300, 0, 81], 5, True, "fp16"),
    (5, 1, 160, [25, 24, 23, 150], 7, False, "bf16"),     # 24 positions a unit
    (22, 1, 160, [9, 8, 0, 140], 130, True, "bf16"),      # 16 + 6 heads a group
]


def slopes_of(H, alibi):
    """Standard slopes for a power of two of heads, drawn ones otherwise."""
    if not alibi:
        return None, None
    if H & (H - 1) == 0:
        return oracle.alibi_slopes(H), None
    s = np.linspace(0.02, 0.7, H).astype(np.float32)
    return s.astype(np.float64), torch.from_numpy(s).cuda()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "H{}Hk{}d{}n{}P{}{}_{}".format(
    c[0], c[1], c[2], len(c[3]), c[4], "_alibi" if c[5] else "", c[6]))
def test_packed_matches_oracle(case):
    H, Hk, d, lens, P, alibi, dt = case
    front, back = 3, 140  # rows of no prompt, poisoned
    cu = ends(lens, front)
    T = cu[-1] + back
    q, k, v, kp, vp = inputs(H, Hk, T, d, P, dt, 900 + H + d + P + T)
    qd, kd, vd = to_dev(q), to_dev(k), to_dev(v)
    for t in (qd, kd, vd):
        t[:, :front] = float("nan")
        t[:, cu[-1]:] = float("inf")
    out = torch.full((T, H, d), 7.0, dtype=qd.dtype, device="cuda")
    ref_slopes, dev_slopes = slopes_of(H, alibi)
    blk.attn_prefill_packed(qd, kd, vd, table(cu), k_prefix=to_dev(kp), v_prefix=to_dev(vp),
                            alibi=alibi, slopes=dev_slopes, out=out)
    blk.check_device_status()
    for i, n in enumerate(lens):
        if n:
            ref = reference(q, k, v, cu[i], n, kp, vp, ref_slopes)
            check_rows(out[cu[i]:cu[i + 1]], ref, dt, f"{case} prompt {i}")
    assert (out[:front] == 7).all() and (out[cu[-1]:] == 7).all()


@pytest.mark.parametrize("H,Hk,d", [(2, 2, 64), (2, 2, 128), (4, 1, 128), (4, 2, 160)])
def test_equal_lengths_equal_the_dense_kernel(H, Hk, d):
    """Prompts of one length are blk_attn_prefill's batch: at head_dim 64 bit for
    bit (the same products in the same order); above, where the packed kernel's
    key tiles are narrower, to the roundings of P and o on either side."""
    B, S = 3, 333
    q, k, v, _, _ = inputs(H, Hk, B * S, d, 0, "bf16", 71)
    qd, kd, vd = to_dev(q), to_dev(k), to_dev(v)
    o = blk.attn_prefill_packed(qd, kd, vd, table(ends([S] * B)))
    dense = blk.attn_prefill(*(t.view(t.shape[0], B, S, d).transpose(0, 1).contiguous() for t in (qd, kd, vd)))
    if d == 64:
        assert torch.equal(o.view(B, S, H, d), dense)
    for b in range(B):
        ref = reference(q, k, v, b * S, S)
        check_rows(o[b * S:(b + 1) * S], ref, "bf16", f"packed, prompt {b}")
        check_rows(dense[b], ref, "bf16", f"dense, prompt {b}")


@pytest.mark.parametrize("H,Hk,d,P", [(2, 2, 64, 0), (2, 2, 128, 70), (4, 1, 128, 0), (4, 1, 160, 300)])
def test_prompts_do_not_touch_each_other(H, Hk, d, P):
    """A prompt full of NaN and infinities leaves the others' bits alone."""
    lens = [100, 57, 300, 1]
    cu = ends(lens)
    q, k, v, kp, vp = inputs(H, Hk, cu[-1], d, P, "bf16", 5)
    qd, kd, vd = to_dev(q), to_dev(k), to_dev(v)
    args = dict(k_prefix=to_dev(kp), v_prefix=to_dev(vp))
    good = blk.attn_prefill_packed(qd, kd, vd, table(cu), **args)
    for i in (1, 3):
        for t, bad in ((qd, float("nan")), (kd, float("inf")), (vd, float("nan"))):
            t[:, cu[i]:cu[i + 1]] = bad
    o = blk.attn_prefill_packed(qd, kd, vd, table(cu), **args)
    for i in (0, 2):
        assert torch.equal(o[cu[i]:cu[i + 1]], good[cu[i]:cu[i + 1]])


@pytest.mark.parametrize("H,Hk,d", [(2, 2, 64), (2, 2, 128), (4, 1, 128), (4, 1, 160)])
def test_list_in_the_workspace(H, Hk, d):
    """The same prompts, and empty ones behind them that make the table too
    long for the CTAs' own lists: the same bits."""
    lens = [100, 257, 300, 1, 513]
    cu = ends(lens)
    q, k, v, kp, vp = inputs(H, Hk, cu[-1], d, 150, "bf16", 17)
    args = to_dev(q), to_dev(k), to_dev(v)
    pre = dict(k_prefix=to_dev(kp), v_prefix=to_dev(vp))
    a = blk.attn_prefill_packed(*args, table(cu), **pre)
    b = blk.attn_prefill_packed(*args, table(cu + [cu[-1]] * 300), **pre)
    assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128, 160])
def test_growing_scores_rescale(d):
    """Keys whose scores rise along the prompt move the running maximum at
    every tile, the prefix's among them."""
    H, n, P = 2, 500, 200
    q, k, v, kp, vp = inputs(H, H, n, d, P, "bf16", 8)
    ramp = torch.linspace(0.0, 3.0, P + n)
    q = torch.ones_like(q)
    k = (ramp[P:, None] * torch.ones(H, n, d)).to(torch.bfloat16)
    kp = (ramp[:P, None] * torch.ones(H, P, d)).to(torch.bfloat16)
    o = blk.attn_prefill_packed(to_dev(q), to_dev(k), to_dev(v), table([0, n]), k_prefix=to_dev(kp),
                                v_prefix=to_dev(vp))
    check_rows(o, reference(q, k, v, 0, n, kp, vp), "bf16", f"d {d}")


def test_all_prompts_empty():
    q, k, v, _, _ = inputs(2, 2, 40, 64, 0, "bf16", 3)
    out = torch.full((40, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    blk.attn_prefill_packed(to_dev(q), to_dev(k), to_dev(v), table([7, 7, 7]), out=out)
    blk.check_device_status()
    assert (out == 5).all()


def test_table_is_clamped():
    """Entries outside [0, tokens], or falling, read and write nothing outside
    the tensors: the prompts they make are cut to them."""
    q, k, v, _, _ = inputs(2, 2, 300, 64, 0, "bf16", 4)
    args = to_dev(q), to_dev(k), to_dev(v)
    o = blk.attn_prefill_packed(*args, table([-9, 100, 100000]))
    want = blk.attn_prefill_packed(*args, table([0, 100, 300]))
    assert torch.equal(o, want)
    o = blk.attn_prefill_packed(*args, table([0, 300, 5, 5]))  # 300 > 5: an empty prompt
    blk.check_device_status()
    assert torch.equal(o, blk.attn_prefill_packed(*args, table([0, 300])))


@pytest.mark.parametrize("prompts", [700, 5000])
def test_long_table_that_overlaps(prompts):
    """A long table that goes up and down between the ends, as if every other
    prompt had all rows, makes no more work than the rows have: the list, in the
    workspace, takes each entry as at least the greatest before it."""
    T = 520
    q, k, v, _, _ = inputs(2, 2, T, 64, 0, "bf16", 4)
    args = to_dev(q), to_dev(k), to_dev(v)
    bad = [(0, T, 0, 2 * T, -T)[i % 5] for i in range(prompts + 1)]
    out = torch.full((T, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    blk.attn_prefill_packed(*args, table(bad), out=out)
    blk.check_device_status()
    assert torch.equal(out, blk.attn_prefill_packed(*args, table([0, T])))
    # and rising entries between falling ones: 0, 100, 50, 300, 200, 300, ...
    want = blk.attn_prefill_packed(*args, table([0, 100, 300]), out=torch.full_like(out, 3.0))
    got = blk.attn_prefill_packed(*args, table([0, 100, 50] + [300, 200] * (prompts // 2)),
                                  out=torch.full_like(out, 3.0))
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2049])
def test_list_in_pieces(n):
    """Tables whose prompts end at and around the pieces the list is made of."""
    lens = [1 + (i % 3 == 0) for i in range(n - 1)] + [260]
    cu = ends(lens)
    q, k, v, _, _ = inputs(1, 1, cu[-1], 64, 0, "fp16", 9)
    o = blk.attn_prefill_packed(to_dev(q), to_dev(k), to_dev(v), table(cu))
    assert torch.equal(o[0], to_dev(v)[0, :1])   # one visible key: its value row
    for i in (1, 2, 1021, 1022, 1023, 1024, n - 2, n - 1):
        if i < n:
            check_rows(o[cu[i]:cu[i + 1]], reference(q, k, v, cu[i], lens[i]), "fp16", f"prompt {i}")


@pytest.mark.parametrize("prompts", [255, 700])
def test_many_prompts(prompts):
    """Many prompts of a few tokens, the list built by each CTA (up to 256) or
    in the workspace."""
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 5, prompts)] + [300]
    cu = ends(lens)
    q, k, v, _, _ = inputs(2, 1, cu[-1], 64, 0, "fp16", 6)
    o = blk.attn_prefill_packed(to_dev(q), to_dev(k), to_dev(v), table(cu), alibi=True)
    for i, n in enumerate(lens):
        if n:
            check_rows(o[cu[i]:cu[i + 1]], reference(q, k, v, cu[i], n, slopes=oracle.alibi_slopes(2)),
                       "fp16", f"prompt {i}")


def test_scale_and_slopes():
    q, k, v, _, _ = inputs(3, 3, 200, 64, 0, "bf16", 9)
    s = np.array([0.5, 0.01, 0.0], dtype=np.float32)
    o = blk.attn_prefill_packed(to_dev(q), to_dev(k), to_dev(v), table([0, 77, 200]), alibi=True,
                                slopes=torch.from_numpy(s).cuda(), scale=0.3)
    for a, b in ((0, 77), (77, 200)):
        check_rows(o[a:b], reference(q, k, v, a, b - a, slopes=s.astype(np.float64), scale=np.float32(0.3)),
                   "bf16", "scale and slopes")


def test_graph_replay_and_other_stream():
    """A captured call follows new tables and inputs; a side stream gives the
    same bits."""
    q, k, v, kp, vp = inputs(8, 2, 600, 128, 140, "bf16", 12)
    qd, kd, vd, kpd, vpd = map(to_dev, (q, k, v, kp, vp))
    cu = table([0, 250, 251, 600])
    ws = torch.empty(blk.attn_prefill_packed_workspace_size(blk.packed_desc(600, 3, 8, 2, 128, 140)),
                     dtype=torch.uint8, device="cuda")
    assert ws.numel() == 0
    out = torch.zeros((600, 8, 128), dtype=torch.bfloat16, device="cuda")

    def call():
        return blk.attn_prefill_packed(qd, kd, vd, cu, k_prefix=kpd, v_prefix=vpd, out=out, workspace=ws)

    first = call().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
        assert torch.equal(out, first)
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.synchronize()
    for tab in ([0, 10, 400, 600], [0, 600, 600, 600]):
        cu.copy_(table(tab))
        qd.copy_(qd.flip(1))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, blk.attn_prefill_packed(qd, kd, vd, cu, k_prefix=kpd, v_prefix=vpd))


# ---- the block over packed prompts ------------------------------------

BLOCKS = {
    "stablelm": scaled(BLOCK_CONFIGS["stablelm2_1p6b"], batch=1, hidden=256, n_heads=4, n_kv_heads=4,
                       intermediate=688),
    "bloom": scaled(BLOCK_CONFIGS["bloom_560m"], batch=1, hidden=256, n_heads=4, n_kv_heads=4,
                    intermediate=1024),
    "olmo": scaled(BLOCK_CONFIGS["olmo2_1b"], batch=1, hidden=256, n_heads=2, n_kv_heads=2,
                   intermediate=512),
    "stablelm_12b": scaled(BLOCK_CONFIGS["stablelm2_12b"], batch=1, hidden=320, n_heads=8, n_kv_heads=2,
                           intermediate=512),
}


@pytest.mark.parametrize("name", sorted(BLOCKS))
@pytest.mark.parametrize("extra", [0, 300])
def test_block_over_packed_prompts(name, extra):
    """blk_forward_packed is the oracle's block on each prompt by itself (its
    own positions from 0), at the gates of the block's dense tests, with the
    work list in shared memory or (extra empty prompts) in the workspace."""
    lens = [70, 1, 0, 200, 129]
    cu = ends(lens)
    T = cu[-1] + 5
    cfg = dataclasses.replace(BLOCKS[name], seq=T)
    x, w = workloads.block_inputs(cfg)
    x = x.reshape(T, cfg.hidden)
    wd = {k: to_dev(t) for k, t in w.items()}
    y = blk.forward_packed(cfg, wd, to_dev(x), table(cu + [cu[-1]] * extra))
    blk.check_device_status()
    tol = POST_NORM_ABS_TOL if cfg.norm_place == "post" else ABS_TOL
    for i, n in enumerate(lens):
        if n:
            one = dataclasses.replace(cfg, seq=n)
            ref = oracle.block_forward(one, x[None, cu[i]:cu[i + 1]], w)["y"][0]
            check(y[cu[i]:cu[i + 1]], ref, f"{name} prompt {i}", unit_scale=True, abs_tol=tol,
                  storage=cfg.dtype)


def test_block_over_one_prompt_equals_dense():
    """One prompt that is all rows: the block's dense forward, bit for bit."""
    cfg = dataclasses.replace(BLOCKS["stablelm"], seq=333)
    x, w = workloads.block_inputs(cfg)
    wd = {k: to_dev(t) for k, t in w.items()}
    dense = blk.forward(cfg, wd, to_dev(x))
    y = blk.forward_packed(cfg, wd, to_dev(x)[0], table([0, 333]))
    assert torch.equal(y, dense[0])


def test_captured_without_a_workspace():
    """A captured call with a long list keeps it in the graph's memory."""
    cu = ends([3] * 300 + [200])
    args = [to_dev(t) for t in inputs(2, 1, cu[-1], 64, 0, "bf16", 12)[:3]] + [table(cu)]
    want = blk.attn_prefill_packed(*args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = blk.attn_prefill_packed(*args)
    for _ in range(3):
        o.zero_()
        g.replay()
        blk.attn_prefill_packed(args[0].flip(1).contiguous(), *args[1:])
        torch.cuda.synchronize()
        assert torch.equal(o, want)


def test_binding_refuses():
    q, k, v, kp, vp = (to_dev(t) for t in inputs(4, 2, 64, 64, 32, "bf16", 13))
    cu = table([0, 64])
    with pytest.raises(ValueError):
        blk.attn_prefill_packed(q, k[:, :60], v, cu)
    with pytest.raises(ValueError):
        blk.attn_prefill_packed(q, k, v, cu, k_prefix=kp)
    with pytest.raises(ValueError):
        blk.attn_prefill_packed(q, k, v, cu, k_prefix=kp, v_prefix=vp[:1])
    with pytest.raises(ValueError):
        blk.attn_prefill_packed(q.transpose(0, 1), k, v, cu)
    with pytest.raises(TypeError):
        blk.attn_prefill_packed(q, k.half(), v, cu)
    with pytest.raises(TypeError):
        blk.attn_prefill_packed(q, k, v, cu.long())
    with pytest.raises(ValueError):
        blk.attn_prefill_packed(q, k, v, cu[:1])
    with pytest.raises(ValueError):
        blk.attn_prefill_packed(q, k, v, cu, out=q)
    with pytest.raises(blk.BlkError):
        blk.attn_prefill_packed(q, k, v, torch.zeros(400, dtype=torch.int32, device="cuda"),
                                workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(blk.BlkError):
        blk.attn_prefill_packed(q, k, v, cu, slopes=torch.ones(4, device="cuda"))
