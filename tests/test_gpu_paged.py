"""GPU parity of the decode step over a paged cache (blk_attn_decode_paged) with its
definition in 64 bits, through the Python binding.

Error of one output element (u: half a step of the storage type, relative; n keys):
- 16-bit cache: weights rounded to the storage type, the output once, the 32-bit parts
  (scores, exponentials, sums, merge) less than 2^-13:
    (u + 2^-13) sum p |v| + u |o| + n 2^-25 max |v|
- e4m3: a weight is a sum of two (bf16) or three (fp16) e4m3 numbers: w = 2^-9 or 2^-14 off,
  relative, or, absolute, half a step of the smallest part, 2^-10 2^-5 or 2^-10 2^-10, where the
  largest weight times scale is 64 at least: 2^-21 or 2^-26 of it; the queries' parts are 2^-22
  or less of the row's largest off, so a score at most 2^-22 scale max|q| sum|k|, which is a relative
  error of its weight, twice (weight and sum):
    (w + 2^-13 + e) sum p |v| + u |o| + n 2^-21 (2^-26) max(p scale_v) 448
"""
import numpy as np
import pytest
import torch

import alibi_attention_block_gb300 as blk
from tests import paged_ref as ref
from tests.parity import f64
from tests.test_gpu_packed import slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(pages, Hk, n, d, dt, bits, g, spread=0.0):
    """Random caches [pages, Hk, n, d]: (k, v, k_scale, v_scale); spread: binary orders of
    magnitude over which pages' scales vary."""
    out, scales = [], []
    for _ in "kv":
        x = torch.randn((pages, Hk, n, d), generator=g, device="cuda") + 0.3
        if bits == 16:
            out.append(x.to(ref.DTYPES[dt]))
            scales.append(None)
        else:
            s = torch.exp2(-7 + torch.randint(0, 2, (pages, Hk), generator=g, device="cuda").float())
            out.append((x / s[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn))
            if spread:
                s = s * torch.exp2(spread * (torch.rand((pages, Hk), generator=g, device="cuda") - 0.5))
            scales.append(s)
    return out[0], out[1], scales[0], scales[1]


def check(got, q, k, v, ks, vs, table, lens, page, dt, slopes=None, scale=None, name=""):
    u = ref.HALF_STEP[dt]
    e8 = ks is not None
    got, qd = f64(got.float()), f64(q.float())
    for b, n in enumerate(lens):
        n = max(0, min(n, table.shape[1] * page))
        if n == 0:
            assert not got[b].any(), f"{name} row {b} is not zero"
            continue
        tb = table[b].tolist()
        kr, seen, _ = ref.rows(k, ks, tb, n, page)
        vr, _, sc = ref.rows(v, vs, tb, n, page)
        o, mag, p = ref.decode(qd[b], kr, vr, seen, slopes, scale)
        if not seen.any():
            assert not got[b].any(), f"{name} row {b} is not zero"
            continue
        grp = qd.shape[1] // kr.shape[0]
        if e8:
            w, tiny = (2.0 ** -9, 2.0 ** -21) if dt == "bf16" else (2.0 ** -14, 2.0 ** -26)
            sm = kr.shape[2] ** -0.5 if scale is None else scale
            e = 2 * 2.0 ** -22 * sm * np.abs(qd[b]).max(1) * np.abs(np.repeat(kr, grp, 0)).sum(2).max(1)
            low = n * tiny * 448 * (p * np.repeat(sc, grp, 0)).max(1)
            bound = (w + 2.0 ** -13 + e[:, None]) * mag + u * np.abs(o) + low[:, None]
        else:
            bound = (u + 2.0 ** -13) * mag + u * np.abs(o) + n * 2.0 ** -25 * np.abs(vr).max()
        err = np.abs(got[b] - o)
        assert np.isfinite(got[b]).all(), f"{name} row {b}: non-finite output"
        assert (err <= bound).all(), \
            f"{name} row {b}: error {err.max():.3e}, {float((err / bound).max()):.2f} of the bound"


def run(B, H, Hk, d, page, lens, dt, bits, alibi=False, seed=0, spread=0.0, scale=None, room=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    k, v, ks, vs = pool(pages, Hk, page, d, dt, bits, g, spread)
    table = torch.full((B, max(need) + room), -1, dtype=torch.int32)
    order = np.random.RandomState(seed).permutation(pages)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(order[at:at + m].astype(np.int32))
        at += m
    # what lies behind a sequence's end is not part of it
    nan = 0x7F if bits == 8 else {"bf16": 0x7FC0, "fp16": 0x7E00}[dt]
    for b, n in enumerate(lens):
        if n % page:
            for c in (k, v):
                c.view(torch.uint8 if bits == 8 else torch.int16)[int(table[b, n // page]), :, n % page:] = nan
    q = torch.randn((B, H, d), generator=g, device="cuda").to(ref.DTYPES[dt])
    ref_slopes, dev_slopes = slopes_of(H, alibi)
    o = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens), k_scale=ks, v_scale=vs, alibi=alibi,
                              slopes=dev_slopes, scale=scale)
    blk.check_device_status()
    check(o, q, k, v, ks, vs, table, lens, page, dt, ref_slopes, scale, name=f"{(B, H, Hk, d, page, dt, bits)}")


CASES = [
    # B, H, Hk, d, page, lens, alibi
    (1, 1, 1, 128, 16, [1], False),
    (1, 4, 1, 128, 128, [128], False),
    (2, 2, 2, 64, 16, [17, 0], True),
    (3, 8, 2, 128, 64, [200, 1, 129], False),
    (2, 8, 1, 64, 32, [300, 127], True),
    (2, 4, 1, 160, 32, [257, 33], False),
    (2, 2, 2, 160, 128, [127, 500], True),
    (5, 16, 2, 160, 16, [1, 2, 15, 16, 640], False),
    (3, 6, 2, 128, 32, [100, 31, 1000], False),     # groups of 3
    (2, 5, 1, 64, 64, [90, 700], False),            # of 5
    (2, 7, 1, 128, 16, [140, 47], False),           # of 7
    (2, 24, 2, 128, 64, [77, 513], True),           # of 12: two units
    (2, 32, 1, 64, 16, [130, 5], False),            # all heads on one
    (70, 4, 4, 64, 16, [(37 * i) % 300 for i in range(70)], False),
    (300, 2, 1, 128, 16, [i % 40 for i in range(300)], True),
    (2, 8, 2, 128, 64, [20000, 3], False),
]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 160])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_every_kernel(G, d, dt, bits):
    """Each instantiation with more tiles than CTAs: several segments each, of several tiles,
    and tails of every kind; with ALiBi too."""
    lens = [(211 * i) % 1700 for i in range(27)]
    for alibi in (False, True):
        run(27, 4 * G, 4, d, 32, lens, dt, bits, alibi, seed=G + d, spread=6.0 if alibi else 0.0)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}H{}Hk{}d{}p{}".format(*c[:5]))
def test_matches_definition(case, dt, bits):
    """With room to spare in the block table, every case takes the two launches."""
    B, H, Hk, d, page, lens, alibi = case
    for room in (0, 2000):
        run(B, H, Hk, d, page, lens, dt, bits, alibi, seed=B + H + d, room=room)


def test_room_chooses_the_form():
    def need(max_pages, page):
        return blk.attn_decode_paged_workspace_size(blk.decode_paged_desc(
            (9, page, 2, 64, 3, max_pages, 2 * page * 64, 1), 4, 256, 64))
    assert need(32, 16) == 0 and need(4, 128) == 0 and need(33, 16) > 0 and need(5, 128) > 0
