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
        # below its normal range (2^-14, fp16) the type's steps are 2^-24: half of one, 2^-25, whatever the value
        bound = bound + {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}[dt]
        # a value of 65520 and more has no fp16 number: it rounds to the infinity of its sign
        over = (dt == "fp16") & (np.abs(o) + bound >= 65520.0) & np.isinf(got[b]) & (np.sign(got[b]) == np.sign(o))
        err = np.where(over, 0.0, np.abs(np.where(over, 0.0, got[b]) - o * ~over))
        assert (np.isfinite(got[b]) | over).all(), f"{name} row {b}: non-finite output"
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
@pytest.mark.parametrize("d", [64, 128, 160])
@pytest.mark.parametrize("G", [9, 16, 17, 40])
def test_many_heads_of_a_kv_head(G, d, dt, bits):
    """More than eight query heads on a kv head, the last unit full, part empty or of one head:
    with several segments per CTA, and in one launch; with ALiBi too."""
    lens = [(211 * i) % 1700 for i in range(27)]
    run(27, 3 * G, 3, d, 32, lens, dt, bits, True, seed=G + d, spread=6.0)
    run(27, 3 * G, 3, d, 64, lens, dt, bits, False, seed=G + d + 1)
    run(9, 2 * G, 2, d, 16, [(53 * i) % 400 for i in range(9)], dt, bits, True, seed=G + d + 2, spread=6.0)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("d,H,Hk", [(64, 2, 2), (128, 8, 1), (160, 4, 1)])
@pytest.mark.parametrize("B", [1, 5, 700])
def test_one_long_sequence(B, d, H, Hk, bits):
    """A row joined from nearly every CTA's part of it, alone and among many rows of one part or none."""
    lens = [i % 9 for i in range(B)]
    lens[B // 2] = 50003
    run(B, H, Hk, d, 64, lens, "fp16", bits, B == 5, seed=B + d)


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


@pytest.mark.parametrize("d,Hk,G", [(64, 2, 1), (128, 2, 4), (160, 1, 8)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_scales_of_any_size(d, Hk, G, dt):
    """Scales that are no powers of two, and over 40 binary orders: the weights' reference goes by
    score + log2(scale)."""
    run(4, Hk * G, Hk, d, 16, [700, 90, 16, 1300], dt, 8, seed=d, spread=40.0, room=100)
    run(4, Hk * G, Hk, d, 16, [300, 90, 16, 500], dt, 8, True, seed=d, spread=20.0, room=0, scale=0.3)


def simple(B, Hk, G, d, page, pages, dt="bf16", bits=8, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    k, v, ks, vs = pool(pages, Hk, page, d, dt, bits, g)
    q = torch.randn((B, Hk * G, d), generator=g, device="cuda").to(ref.DTYPES[dt])
    return q, k, v, ks, vs


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("room", [0, 60])
def test_pages_that_are_not_there(room, bits):
    """Keys in pages outside the pool take no part (their rows hold NaN codes elsewhere), a row without any is zero;
    a page may occur twice, and in two sequences."""
    page, n = 16, 300
    q, k, v, ks, vs = simple(5, 2, 4, 128, page, 40, bits=bits)
    table = torch.arange(5 * 19, dtype=torch.int32).reshape(5, 19) % 40
    table[0, 3], table[0, 18], table[1, 5:14] = -1, 40, 2 ** 31 - 1
    table[2] = -2 ** 31                          # none at all
    table[3, :9] = 999                           # the oldest tiles: nothing seen in them
    table[4, 8:] = 77                            # the newest tiles: nothing seen at first
    table = torch.cat((table, torch.full((5, room), -1, dtype=torch.int32)), 1)
    lens = [n, n, n, n, n]
    o = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens), k_scale=ks, v_scale=vs)
    blk.check_device_status()
    check(o, q, k, v, ks, vs, table, lens, page, "bf16")
    assert not o[2].any()


def test_lengths_that_do_not_fit():
    page = 32
    q, k, v, ks, vs = simple(4, 1, 2, 64, page, 9, seed=1)
    table = (torch.arange(4 * 6, dtype=torch.int32) % 9).reshape(4, 6)
    lens = [10 ** 6, -5, 0, 2 ** 31 - 1]
    for room in (0, 20):
        t = torch.cat((table, torch.full((4, room), -1, dtype=torch.int32)), 1)
        o = blk.attn_decode_paged(q, k, v, t.cuda(), i32(lens), k_scale=ks, v_scale=vs)
        check(o, q, k, v, ks, vs, t, lens, page, "bf16")


@pytest.mark.parametrize("room", [0, 60])
@pytest.mark.parametrize("bits", [8, 16])
def test_not_finite_numbers(room, bits):
    """A NaN in a key or value reaches its kv head's rows, one in a query its head, and no other; a
    masked one (behind the length, covered elsewhere) none."""
    page = 16
    q, k, v, ks, vs = simple(4, 2, 4, 64, page, 64, bits=bits, seed=2)
    table = torch.arange(4 * 16, dtype=torch.int32).reshape(4, 16)
    table = torch.cat((table, torch.full((4, room), -1, dtype=torch.int32)), 1)
    lens = [250, 200, 129, 40]
    good = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens), k_scale=ks, v_scale=vs)
    nan = torch.tensor(float("nan")).to(k.dtype)
    k, v, q = k.clone(), v.clone(), q.clone()
    view = lambda x: x.view(torch.uint8) if bits == 8 else x  # noqa: E731
    bad = nan.view(torch.uint8) if bits == 8 else nan
    view(k)[0, 1, 5, 7] = bad
    view(v)[16 + 11, 0, 3, 9] = bad
    q[2, 6, 30] = float("nan")
    q[3, 1, 2] = float("inf")
    o = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens), k_scale=ks, v_scale=vs)
    where = torch.zeros_like(o, dtype=torch.bool)
    where[0, 4:] = True          # a key's NaN: its kv head
    where[1, :4, 9] = True       # a value's: its kv head's dim
    where[2, 6] = True
    where[3, 1] = True
    assert torch.equal(torch.isnan(o), where)
    assert torch.equal(o[~where], good[~where])


def test_large_scores():
    """Scores over a wide range, growing and falling along the cache: the reference moves many times."""
    for dt in ("bf16", "fp16"):
        for bits in (8, 16):
            page, n = 64, 3000
            q, k, v, ks, vs = simple(2, 2, 4, 128, page, 100, dt, bits, seed=3)
            rise = torch.linspace(-1, 1, 48, device="cuda")[:, None, None, None]
            far = (k.float()[:96] * 0.2 + torch.cat((rise, -rise)) * q[0, 0].float() / 4).to(k.dtype)
            k[:96].copy_(far) if bits == 16 else k.view(torch.uint8)[:96].copy_(far.view(torch.uint8))
            if bits == 8:
                ks.fill_(0.25)
            table = torch.arange(96, dtype=torch.int32).reshape(2, 48)
            o = blk.attn_decode_paged(q, k, v, table.cuda(), i32([n, n - 77]), k_scale=ks, v_scale=vs)
            check(o, q, k, v, ks, vs, table, [n, n - 77], page, dt, name=f"{dt} {bits}")


def test_streams_graphs_and_views():
    """The same bits twice; on two streams at once, each with a workspace; captured, with lengths and table
    changed between replays; from views (one pool for keys and values, strided queries, given out)."""
    B, Hk, G, d, page = 6, 2, 4, 128, 32
    q, k, v, ks, vs = simple(B, Hk, G, d, page, 200, seed=4)
    table = torch.arange(6 * 33, dtype=torch.int32).reshape(6, 33).cuda()
    lens = i32([1000, 3, 0, 517, 128, 1056])

    def call(**kw):
        return blk.attn_decode_paged(q, k, v, table, lens, k_scale=ks, v_scale=vs, **kw)
    a = call()
    assert torch.equal(a, call())
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for o in outs)
    both = torch.stack((k.view(torch.uint8), v.view(torch.uint8)), 1).view(torch.float8_e4m3fn)
    wide = torch.zeros((Hk * G, B, d + 8), dtype=q.dtype, device="cuda")
    wide[..., :d] = q.transpose(0, 1)
    out = torch.empty_like(q)
    got = blk.attn_decode_paged(wide[..., :d].transpose(0, 1), both[:, 0], both[:, 1], table, lens, k_scale=ks, v_scale=vs,
                                out=out)
    assert got is out and torch.equal(out, a)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    graph, o = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        call(out=o, workspace=ws)
    for new in ([5, 0, 999, 1, 31, 640], [0] * 6, [1056] * 6):
        lens.copy_(i32(new))
        table.copy_(table.flip(0))
        ws.fill_(0xFF)  # what a workspace holds before does not matter
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, call())
        check(o, q, k, v, ks, vs, table.cpu(), new, page, "bf16")
    blk.check_device_status()


def test_workspace_of_one_alignment():
    """Workspaces at every multiple of 16 bytes, with nothing written around them."""
    q, k, v, ks, vs = simple(3, 2, 1, 160, 16, 120, seed=5)
    table = torch.arange(3 * 40, dtype=torch.int32).reshape(3, 40).cuda()
    lens = i32([640, 5, 333])
    need = blk.attn_decode_paged_workspace_size(blk.decode_paged_desc((120, 16, 2, 160, 3, 40, 2 * 16 * 160, 1), 2, 320, 160))
    a = blk.attn_decode_paged(q, k, v, table, lens, k_scale=ks, v_scale=vs)
    for at in (16, 32, 48, 240):
        buf = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        o = blk.attn_decode_paged(q, k, v, table, lens, k_scale=ks, v_scale=vs, workspace=buf[at:at + need])
        assert torch.equal(o, a)
        assert bool((buf[:at] == 0xA5).all()) and bool((buf[at + need:] == 0xA5).all())


def test_many_sequences():
    """More sequences than threads that sum them, most of them short or away."""
    B, page = 3000, 16
    q, k, v, ks, vs = simple(B, 1, 1, 64, page, 500, seed=6)
    lens = [(7 * i) % 50 if i % 3 else 0 for i in range(B)]
    table = (torch.arange(B * 40, dtype=torch.int32) * 7 % 500).reshape(B, 40)
    o = blk.attn_decode_paged(q, k, v, table.cuda(), i32(lens), k_scale=ks, v_scale=vs)
    pick = list(range(0, B, 37))
    check(o[pick], q[pick], k, v, ks, vs, table[pick], [lens[b] for b in pick], page, "bf16")
    assert not o[[b for b in range(B) if lens[b] == 0]].any()
