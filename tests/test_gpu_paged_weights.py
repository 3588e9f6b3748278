"""The softmax weights of the paged decode step (blk_attn_decode_paged), as exact as the 32 bits
that they are computed in, but for what their parts leave: with few keys an output does not
average the weights' errors.

Error of one output element (u: half a step of the storage type, relative; A: the largest over the keys of
scale log2(e) sum |q_i k_i|):
- a weight's parts, w: two bf16 numbers, 2^-8 2^-8; two fp16 numbers, 2^-11 2^-11; three e4m3
  numbers, 2^-4 of a half step of the one before each, 2^-5 2^-5 2^-4 (each part's remainder is at most
  2^-5 of the range that it lies in);
- a score: d products added in steps of 16 or more, each step 2^-24 of what is there, and five
  32-bit factors, 2^-24 each: (160 / 16 + 2 + 5) 2^-24 A < 2^-19 A; less the reference, 2^-24 2 A; its exponential 2^-22:
  a weight's relative error is ln(2) (2^-19 + 2^-23) A + 2^-22 =: e, once in the sum with V and once in the weights' sum;
- sums of up to 2^9 steps in 32 bits, the merge's exponentials and the division: less than 2^-14 2^-5 = 2^-19 by far for
  the few hundred keys here;
- e4m3: the parts' least half step, 2^-10 2^-10 of where the largest weight times scale is 64 at least: 2^-26 of it
  for each key; and the queries' parts, 2^-22 of the row's largest, as in test_gpu_paged.py;
- the output's rounding, u (and half of the type's least step).
  (w + 2 e + 2^-19) sum p |v| + u |o| [+ n 2^-26 max(p scale_v) 448]
"""
import math

import numpy as np
import pytest
import torch

import alibi_attention_block_gb300 as blk
from tests import paged_ref as ref
from tests.parity import f64

pytestmark = pytest.mark.gpu
PARTS = {(16, "bf16"): 2.0 ** -16, (16, "fp16"): 2.0 ** -22, (8, "bf16"): 2.0 ** -14, (8, "fp16"): 2.0 ** -14}
LEAST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bound_of(q, kr, vr, sc, o, mag, p, dt, bits, scale):
    """The bound of a row's elements: q [H, d], kr and vr [Hk, n, d], sc [Hk, n] scales of V."""
    grp = q.shape[0] // kr.shape[0]
    kk = np.abs(np.repeat(kr, grp, 0))
    a = (np.abs(q)[:, None] * kk).sum(2).max(1) * scale * math.log2(math.e)
    e = math.log(2) * (2.0 ** -19 + 2.0 ** -23) * a + 2.0 ** -22
    low = 0.0
    if bits == 8:
        e = e + 2.0 ** -22 * scale * np.abs(q).max(1) * kk.sum(2).max(1)
        low = kr.shape[1] * 2.0 ** -26 * 448 * (p * np.repeat(sc, grp, 0)).max(1)[:, None]
    u = ref.HALF_STEP[dt] * (1 + 2.0 ** -10)
    return (PARTS[bits, dt] + 2 * e[:, None] + 2.0 ** -19) * mag + u * np.abs(o) + low + LEAST[dt]


def held(x, bits, dt, scale):
    """x [pages, Hk, n, d] as a cache holds it, at scales [pages, Hk]."""
    if bits == 16:
        return x.to(ref.DTYPES[dt]), None
    return x.clamp(-448, 448).to(torch.float8_e4m3fn), scale.float()


def check(o, q, k, v, ks, vs, table, lens, page, dt, scale=None, name=""):
    bits = 8 if ks is not None else 16
    got, qd = f64(o.float()), f64(q.float())
    s = q.shape[2] ** -0.5 if scale is None else scale
    worst = 0.0
    for b, n in enumerate(lens):
        kr, seen, _ = ref.rows(k, ks, table[b].tolist(), n, page)
        vr, _, sc = ref.rows(v, vs, table[b].tolist(), n, page)
        assert seen.all()
        want, mag, p = ref.decode(qd[b], kr, vr, seen, None, s)
        bound = bound_of(qd[b], kr, vr, sc, want, mag, p, dt, bits, s)
        assert np.isfinite(got[b]).all(), f"{name} row {b}"
        worst = max(worst, float((np.abs(got[b] - want) / bound).max()))
    assert worst <= 1, f"{name}: {worst:.2f} of the bound"


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 160])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
def test_few_keys(G, d, dt, bits):
    """2 to 25 keys, in one launch and in two; two kv heads."""
    B, page, Hk = 24, 16, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(d + G)
    x = [torch.randn((2 * B, Hk, page, d), generator=g, device="cuda") * (1 if bits == 16 else 60) for _ in "kv"]
    (k, ks), (v, vs) = (held(t, bits, dt, torch.full((2 * B, Hk), 2.0 ** -6, device="cuda")) for t in x)
    q = torch.randn((B, Hk * G, d), generator=g, device="cuda").to(ref.DTYPES[dt])
    lens = [2 + b for b in range(B)]
    for room in (0, 60):
        table = torch.full((B, 2 + room), -1, dtype=torch.int32)
        table[:, :2] = torch.arange(2 * B, dtype=torch.int32).reshape(B, 2)
        o = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens), k_scale=ks, v_scale=vs)
        check(o, q, k, v, ks, vs, table, lens, page, dt, name=f"room {room}")
    blk.check_device_status()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,n", [(3, 512), (400, 2000)])
def test_many_small_weights(B, n, d, dt):
    """A key whose value is 0 far above equal ones of 2^-20.375 of its weight, which are all of the output: 16-bit caches, in
    one launch, and with whole sequences to a CTA in two (all over the same pages). 2^-20.375 is no number of fp16's
    least steps, 2^-24; its roundings are all alike."""
    page = 128
    pages = -(-n // page)
    t = ref.DTYPES[dt]
    k, v = torch.zeros((pages, 1, page, d), device="cuda", dtype=t), torch.ones((pages, 1, page, d), device="cuda", dtype=t)
    q = torch.zeros((B, 4, d), device="cuda", dtype=t)
    q[..., 0] = 1
    k[(n - 1) // page, 0, (n - 1) % page, 0] = 163  # 20.375 * 8
    v[(n - 1) // page, 0, (n - 1) % page] = 0
    table = torch.arange(pages, dtype=torch.int32).repeat(B, 1)
    scale = math.log(2) / 8
    o = f64(blk.attn_decode_paged(q, k, v, table.cuda(), i32([n] * B), scale=scale).float())
    w = (n - 1) * 2.0 ** -20.375
    want = w / (1 + w)
    # a score is one product by 32-bit factors: 6 of 2^-24 of 20.4; then as above
    e = math.log(2) * 6 * 2.0 ** -24 * 20.375 + 2.0 ** -22
    bound = (PARTS[16, dt] + 2 * e + 2.0 ** -19 + ref.HALF_STEP[dt] * (1 + 2.0 ** -10)) * want
    worst = np.abs(o - want).max()
    assert worst <= bound, f"{worst / bound:.2f} of the bound"


@pytest.mark.parametrize("d,G", [(64, 1), (128, 4), (160, 8)])
@pytest.mark.parametrize("lo,hi", [(118, 118), (112, 119), (-59, -59), (-60, -50), (-60, 118)])
def test_scales_at_the_ends(lo, hi, d, G):
    """Scales of V of 2^lo to 2^hi, from page to page: those that appended bf16 values take are 2^-60 to 2^120."""
    B, page, Hk = 6, 16, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(d + lo)
    lens = [300, 17, 500, 2, 129, 40]
    k, v = ((torch.randn((200, Hk, page, d), generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            for _ in "kv")
    ks = torch.full((200, Hk), 2.0 ** -6, device="cuda")
    vs = torch.exp2(torch.randint(lo, hi + 1, (200, Hk), generator=g, device="cuda").double()).float()
    q = torch.randn((B, Hk * G, d), generator=g, device="cuda").bfloat16()
    for room in (0, 60):
        table = torch.full((B, 32 + room), -1, dtype=torch.int32)
        table[:, :32] = torch.arange(B * 32, dtype=torch.int32).reshape(B, 32)
        o = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens), k_scale=ks, v_scale=vs)
        check(o, q, k, v, ks, vs, table, lens, page, "bf16", name=f"room {room}")
    blk.check_device_status()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 4), (128, 16), (160, 8)])
@pytest.mark.parametrize("room,times", [(0, 1), (200, 1), (200, 90)])
def test_scores_of_minus_infinity(room, times, d, G, dt):
    """Seen keys whose scores are all -inf leave no softmax: NaN, as the definition's 0 / 0; with a finite one beside
    them they weigh nothing; without any seen key the row is zero. 16 bits, several of a CTA's ranges or one;
    the batch many times over (few rows and many are joined differently)."""
    page, Hk, t = 16, 2, ref.DTYPES[dt]
    B, cols = 8, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(d + G)
    k, v = (torch.randn((B * cols, Hk, page, d), generator=g, device="cuda").to(t) for _ in "kv")
    q = torch.randn((B, Hk * G, d), generator=g, device="cuda").to(t)
    lens = [500, 400, 512, 512, 300, 300, 0, 100]
    table = torch.full((B, cols + room), -1, dtype=torch.int32)
    table[:, :cols] = torch.arange(B * cols, dtype=torch.int32).reshape(B, cols)
    rows = k.view(B, cols, Hk, page, d)
    q[:, :, 0] = 1
    q[0, :, 0] = float("inf")
    rows[0, :, :, :, 0] = -1                    # an infinite query against keys of the other sign
    rows[1, :, :, :, 0] = -float("inf")         # infinite keys, all of them
    rows[2, :16, :, :, 0] = -float("inf")       # the oldest 256
    rows[3, 16:, :, :, 0] = -float("inf")       # the newest 256
    table[4] = 2 ** 30                          # no page is there
    table[5, 3:] = -1                           # those that are there have infinite keys
    rows[5, :, :, :, 0] = -float("inf")
    rows[7, :, :, :, 0] = float("inf")          # +inf - inf: NaN
    o = f64(blk.attn_decode_paged(q.repeat(times, 1, 1), k, v, table.repeat(times, 1).cuda(), i32(lens * times)).float())
    o = o.reshape(times, B, Hk * G, d)
    blk.check_device_status()
    for b in (0, 1, 5, 7):
        assert np.isnan(o[:, b]).all(), f"row {b}"
    assert not o[:, 4].any() and not o[:, 6].any()
    for b, part in ((2, slice(16, 32)), (3, slice(0, 16))):
        kr, vr = (f64(x.view(B, cols, Hk, page, d)[b, part].transpose(0, 1).reshape(Hk, 256, d).float()) for x in (k, v))
        want, mag, p = ref.decode(f64(q[b].float()), kr, vr, np.ones(256, bool))
        bound = bound_of(f64(q[b].float()), kr, vr, None, want, mag, p, dt, 16, d ** -0.5)
        assert (np.abs(o[:, b] - want) <= bound).all(), f"row {b}"


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 4), (128, 16), (160, 8)])
@pytest.mark.parametrize("room", [0, 200])
def test_infinite_values(room, d, G, dt):
    """An infinity among a seen key's values is one in the output (its weight is above 0), whatever the weight's parts are;
    two of both signs are a NaN; a masked key's reach nothing. 16 bits."""
    page, Hk, t = 16, 2, ref.DTYPES[dt]
    B, cols = 4, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(d + G)
    k, v = (torch.randn((B * cols, Hk, page, d), generator=g, device="cuda").to(t) for _ in "kv")
    q = torch.randn((B, Hk * G, d), generator=g, device="cuda").to(t)
    lens = [500, 3, 257, 130]
    table = torch.full((B, cols + room), -1, dtype=torch.int32)
    table[:, :cols] = torch.arange(B * cols, dtype=torch.int32).reshape(B, cols)
    good = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens))
    rows = v.view(B, cols, Hk, page, d)
    want = good.clone().view(B, Hk, G, d)
    inf = float("inf")
    for b, n in enumerate(lens):
        for i, key in enumerate((0, 1, n // 2, n - 2, n - 1)):  # each in a dim of its own; in 20 + i: its negative
            rows[b, key // page, :, key % page, i] = inf
            rows[b, key // page, :, key % page, 20 + i] = -inf
            want[b, :, :, i], want[b, :, :, 20 + i] = inf, -inf
        rows[b, 0, :, 0, 40], rows[b, (n - 1) // page, :, (n - 1) % page, 40] = inf, -inf
        want[b, :, :, 40] = float("nan")
        if n % page:
            rows[b, n // page, :, n % page:] = inf  # behind the length
    o = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens))
    blk.check_device_status()
    want = want.view_as(o)
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    assert torch.equal(o.nan_to_num(7.0, 1e4, -1e4), want.nan_to_num(7.0, 1e4, -1e4))
