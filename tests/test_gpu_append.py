"""GPU parity of rotary at given positions (blk_rope_positions) and of appending to a
paged cache (blk_kv_append_paged) with their definitions in 64 bits.

Turned values: the hardware's sine and cosine are at most 2^-21.2 off between -pi and pi,
their argument 2^-22.3 (24 bits of a half turn, and pi's rounding), the two products
and their sum 2^-23 relative: with x and y the pair, (|x| + |y|) amplitude 2^-20; then
one rounding, u of the value (half of the type's smallest step below its normal range).
"""
import numpy as np
import pytest
import torch

import alibi_attention_block_gb300 as blk
from tests import paged_ref as ref
from tests.parity import f64

pytestmark = pytest.mark.gpu
LEAST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half of the smallest step


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, dt, g):
    return torch.randn(shape, generator=g, device="cuda").to(ref.DTYPES[dt])


def close(got, want, mag, dt, name=""):
    bound = mag * 2.0 ** -20 + ref.HALF_STEP[dt] * np.abs(want) * (1 + 2.0 ** -10) + LEAST[dt]
    err = np.abs(f64(got.float()) - want)
    assert (err <= bound).all(), f"{name}: {float((err / bound).max()):.2f} of the bound"


SCALINGS = [dict(), dict(scaling="linear", factor=4.0),
            dict(scaling="by_parts", factor=8.0, original_len=4096, beta_slow=1.0, beta_fast=32.0)]


@pytest.mark.parametrize("d,span", [(64, 64), (64, 16), (128, 128), (160, 40), (160, 160), (256, 256), (64, 2),
                                    (32, 30), (16, 16), (128, 24)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_rope(d, span, interleaved, dt):
    g = gen(d + span)
    for T, H, Hk, more in ((1, 1, 0, SCALINGS[0]), (37, 4, 2, SCALINGS[1]), (301, 3, 3, SCALINGS[2])):
        amp = 1.25 if more.get("scaling") == "by_parts" else 1.0
        plan = blk.rope_plan(span, 10000.0, interleaved=interleaved, amplitude=amp, **more)
        pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
        pos[0] = 2 ** 31 - 1
        th = ref.thetas(span, 10000.0, **more)
        q = randn((H, T, d), dt, g)
        k = randn((Hk, T, d), dt, g) if Hk else None
        for inverse in (False, True):
            out = blk.rope_positions(q, pos, plan, k=k, inverse=inverse)
            for x, y in ((q, out[0] if Hk else out),) + (((k, out[1]),) if Hk else ()):
                want, mag = ref.turn(f64(x.float()), f64(pos), th, interleaved, amp, inverse)
                # position 2^31 - 1: theta's 53 bits leave 2^-22 of a radian, here and there
                close(y, want, mag * np.where(f64(pos) > 2 ** 30, 3, 1)[None, :, None], dt, f"T{T} inverse {inverse}")
        # in place: the same bits
        q2, k2 = q.clone(), None if k is None else k.clone()
        blk.rope_positions(q2, pos, plan, k=k2, inverse=True, q_out=q2, k_out=k2)
        assert torch.equal(q2, out[0] if Hk else out)
        if Hk:
            assert torch.equal(k2, out[1])


def cache_of(pages, Hk, page, d, dt, bits, g):
    """A pool with old contents everywhere: (k, v, k_scale, v_scale)."""
    shape = (pages, Hk, page, d)
    if bits == 16:
        return randn(shape, dt, g), randn(shape, dt, g), None, None
    codes = [torch.randn(shape, generator=g, device="cuda").mul(90).to(torch.float8_e4m3fn) for _ in "kv"]
    scale = [torch.exp2(torch.randint(-9, -6, (pages, Hk), generator=g, device="cuda").float()) for _ in "kv"]
    return codes[0], codes[1], scale[0], scale[1]


def expect(x, mag, cache, scale, table, before, new, cu, page, dt, got, got_scale, name):
    """One of the caches behind the call: x [Hk, T, d] new values (turned, in 64 bits)."""
    old = cache.cpu().float().double().numpy().copy()
    new_codes = got.cpu().float().double().numpy()
    touched = np.zeros(old.shape[:3], bool)
    s_old = None if scale is None else scale.cpu().double().numpy()
    s_got = None if scale is None else got_scale.cpu().double().numpy()
    seen = set()
    for b, (p0, n) in enumerate(zip(before, new)):
        for j in range(p0 // page, -(-(p0 + n) // page) if n else 0):
            lo, hi = max(p0, j * page), min(p0 + n, (j + 1) * page)
            if j >= table.shape[1] or not 0 <= table[b, j] < old.shape[0]:
                continue
            at, rows = int(table[b, j]), slice(cu[b] + lo - p0, cu[b] + hi - p0)
            off = slice(lo - j * page, hi - j * page)
            touched[at, :, off] = True
            seen.add(at)
            for h in range(x.shape[0]):
                want, m = x[h, rows], mag[h, rows]
                have = new_codes[at, h, off]
                if scale is None:
                    bound = m * 2.0 ** -20 + ref.HALF_STEP[dt] * np.abs(want) * (1 + 2.0 ** -10) + LEAST[dt]
                    assert (np.abs(have - want) <= bound).all(), f"{name} page {at}"
                    continue
                most = np.abs(want).max()
                held = s_old[at, h] if off.start else 0.0
                options = {max(ref.page_scale(y), held) for y in (most - 2.0 ** -20 * m.max(), most, most + 2.0 ** -20 * m.max())}
                s = s_got[at, h]
                assert s in options, f"{name} page {at} head {h}: scale {s}, expected {options}"
                # half a step of e4m3 around the value, and what the turn may be off
                c = np.minimum(np.abs(want / s), 448.0)
                half = np.exp2(np.floor(np.log2(np.maximum(np.maximum(c, np.abs(have)), 2.0 ** -6))) - 4)
                assert (np.abs(have * s - want) <= half * s + m * 2.0 ** -20).all(), f"{name} page {at} head {h}"
                if off.start:
                    r = held / s
                    touched[at, h, :off.start] = True
                    assert np.array_equal(new_codes[at, h, :off.start], ref.e4m3(old[at, h, :off.start] * r),
                                          equal_nan=True), \
                        f"{name} page {at} head {h}: what it held"
    assert np.array_equal(new_codes[~touched], old[~touched], equal_nan=True), f"{name}: other rows changed"
    if scale is not None:
        rest = [i for i in range(old.shape[0]) if i not in seen]
        assert np.array_equal(s_got[rest], s_old[rest]), f"{name}: other scales changed"


def case(H, Hk, d, span, page, before, new, dt, bits, interleaved=False, seed=0, layout="heads", loud=1.0,
         capacity=None, with_q=True, positions=False, one_each=False):
    g = gen(seed)
    T, B = sum(new), len(new)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
    need = [-(-(b + n) // page) for b, n in zip(before, new)]
    pages = sum(need) + 3
    kc, vc, ks, vs = cache_of(pages, Hk, page, d, dt, bits, g)
    table = np.full((B, max(need) if capacity is None else capacity), -1, np.int32)
    order, at = np.random.RandomState(seed).permutation(pages), 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m][:table.shape[1]]
        at += m
    extra = 5  # rows behind the last sequence

    def rows(n):
        x = torch.randn((n, T + extra, d), generator=g, device="cuda") * loud
        x = x.to(ref.DTYPES[dt])
        if layout == "tokens":
            x = x.transpose(0, 1).contiguous().transpose(0, 1)
        return x
    if one_each:
        extra = 0
    k, v, q = rows(Hk), rows(Hk), rows(H) if with_q else None
    plan = blk.rope_plan(span, 10000.0, interleaved=interleaved) if span else None
    at_pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, new)] + [np.zeros(extra)]).astype(np.int64)
    pos = None
    if positions:
        pos = torch.randint(0, 100000, (T + extra,), generator=g, device="cuda", dtype=torch.int32)
        at_pos = f64(pos).astype(np.int64)
    lens = i32([b + n for b, n in zip(before, new)])
    k0, v0 = kc.clone(), vc.clone()
    ks0, vs0 = (None, None) if bits == 16 else (ks.clone(), vs.clone())
    q_out = torch.full_like(q, 7.0) if with_q else None
    out = blk.kv_append_paged(k, v, kc, vc, torch.tensor(table, device="cuda"), lens,
                              cu_seqlens=None if one_each else i32(cu), k_scale=ks, v_scale=vs, rope=plan,
                              positions=pos, q=q, q_out=q_out)
    blk.check_device_status()
    th = ref.thetas(span)
    kt, km = ref.turn(f64(k.float()), at_pos, th, interleaved)
    vf = f64(v.float())
    name = f"{(H, Hk, d, span, page, dt, bits)}"
    expect(kt, km, k0, ks0, table, before, new, cu, page, dt, kc, ks, name + " k")
    expect(vf, 0 * vf, v0, vs0, table, before, new, cu, page, dt, vc, vs, name + " v")
    if with_q:
        qt, qm = ref.turn(f64(q.float()), at_pos, th, interleaved)
        assert out is q_out
        close(out[:, :T], qt[:, :T], qm[:, :T], dt, name + " q")
        assert bool((out[:, T:] == 7.0).all()), "rows behind the last sequence changed"


CASES = [
    # H, Hk, d, span, page, tokens before, new tokens
    (4, 2, 128, 128, 16, [0], [1]),
    (4, 2, 128, 128, 16, [15, 16, 17], [1, 1, 1]),
    (2, 2, 64, 16, 32, [0, 5, 31, 70], [64, 40, 1, 0]),
    (8, 2, 160, 40, 64, [0, 100], [200, 65]),
    (2, 1, 256, 256, 128, [3, 0], [300, 128]),
    (3, 3, 64, 0, 16, [9, 0], [50, 16]),
    (2, 1, 32, 30, 128, [120, 0], [20, 140]),
    (16, 4, 128, 64, 64, [i % 70 for i in range(40)], [(13 * i) % 29 for i in range(40)]),
    (1, 1, 16, 16, 16, [0], [1000]),
]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("c", CASES, ids=lambda c: "H{}Hk{}d{}r{}p{}".format(*c[:5]))
def test_append(c, dt, bits):
    for i, layout in enumerate(("heads", "tokens")):
        case(*c, dt, bits, interleaved=i == 1, seed=c[2] + c[3] + i, layout=layout, loud=1.0 + 3 * i,
             with_q=c[3] > 0)


def test_positions_and_room():
    """Given positions; single tokens without cu_seqlens; pages behind the table and outside the pool."""
    case(4, 2, 128, 128, 32, [0, 40, 7], [33, 30, 0], "bf16", 8, positions=True, seed=1)
    case(4, 2, 64, 64, 16, [0, 15, 16, 100], [1, 1, 1, 1], "fp16", 8, one_each=True, seed=2)
    case(4, 2, 64, 64, 16, [0, 15, 16, 100], [1, 1, 1, 1], "bf16", 16, one_each=True, seed=3)
    case(2, 2, 128, 64, 16, [0, 40], [70, 30], "bf16", 8, capacity=3, seed=4)   # 48 positions of room
    case(2, 2, 128, 64, 16, [0, 40], [70, 30], "bf16", 16, capacity=3, seed=5)


def blank(pages, Hk, page, d, kind):
    dt = torch.float8_e4m3fn if kind == 8 else torch.bfloat16
    caches = [torch.zeros((pages, Hk, page, d), device="cuda").to(dt) for _ in "kv"]
    scales = [torch.full((pages, Hk), 2.0 ** -60, device="cuda") for _ in "kv"] if kind == 8 else [None, None]
    return (*caches, *scales)


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("page", [16, 64])
def test_tokens_one_by_one(page):
    """100 single tokens leave the scales of one call with all of them, and its codes but for those
    that a growing scale has rounded twice (below 2^-6 of it)."""
    Hk, d, n = 3, 64, 100
    g = gen(11)
    k, v = (torch.randn((Hk, n, d), generator=g, device="cuda") * torch.exp2(torch.arange(n, device="cuda") / 9 - 6)[:, None]
            for _ in "kv")
    k, v = k.bfloat16(), v.bfloat16()
    plan = blk.rope_plan(32, 10000.0)
    pages = -(-n // page)
    table = i32([list(range(pages))])
    whole, steps = blank(pages, Hk, page, d, 8), blank(pages, Hk, page, d, 8)
    blk.kv_append_paged(k, v, *whole[:2], table, i32([n]), cu_seqlens=i32([0, n]), k_scale=whole[2], v_scale=whole[3],
                        rope=plan)
    for t in range(n):
        blk.kv_append_paged(k[:, t:t + 1], v[:, t:t + 1], *steps[:2], table, i32([t + 1]), k_scale=steps[2],
                            v_scale=steps[3], rope=plan)
    for i in range(2):
        assert torch.equal(whole[2 + i], steps[2 + i])
        a, b = whole[i].float(), steps[i].float()
        big = a.abs() >= 2.0 ** -6
        assert torch.equal(a[big], b[big])
        assert float((a - b).abs().max()) <= 2.0 ** -9


def test_not_finite_values():
    """NaN stays NaN, an infinity becomes the largest code; the scale is that of the finite values."""
    Hk, d, page = 2, 64, 16
    k = torch.randn((Hk, 20, d), generator=gen(5), device="cuda").bfloat16()
    v = k.clone()
    v[0, 3, 5], v[0, 4, 6], v[0, 5, 7] = float("inf"), -float("inf"), float("nan")
    v[1, 17] = float("inf")  # a page of which ...
    v[1, 16], v[1, 18:] = float("nan"), float("inf")  # ... nothing is finite
    c = blank(2, Hk, page, d, 8)
    blk.kv_append_paged(k, v, *c[:2], i32([[0, 1]]), i32([20]), cu_seqlens=i32([0, 20]), k_scale=c[2], v_scale=c[3])
    got, s = c[1].float(), c[3]
    assert got[0, 0, 3, 5] == 448 and got[0, 0, 4, 6] == -448 and torch.isnan(got[0, 0, 5, 7])
    fin = v[0, :16].float()
    assert float(s[0, 0]) == ref.page_scale(float(fin[torch.isfinite(fin)].abs().max()))
    assert float(s[1, 1]) == 2.0 ** -60 and torch.isnan(got[1, 1, 0]).all() and (got[1, 1, 1:4] == 448).all()
    assert torch.isfinite(got[0, 1]).all() and torch.isfinite(c[0].float()).all()


def test_bits_of_a_call():
    """Twice the same bits; with views of one pool, on another stream, in place, as a graph replayed."""
    Hk, H, d, page, B = 2, 4, 128, 32, 5
    g = gen(6)
    new, before = [40, 1, 0, 70, 33], [0, 31, 5, 10, 64]
    T = sum(new)
    cu, lens = i32(np.concatenate([[0], np.cumsum(new)]).tolist()), i32([a + b for a, b in zip(new, before)])
    table = i32([[5 * j + b for j in range(4)] for b in range(B)])
    k, v, q = (randn((n, T, d), "bf16", g) for n in (Hk, Hk, H))
    plan = blk.rope_plan(128, 500000.0, interleaved=True)

    def run(c, q=q, **kw):
        return blk.kv_append_paged(k, v, c[0], c[1], table, lens, cu_seqlens=cu, k_scale=c[2], v_scale=c[3], rope=plan,
                                   q=q, **kw)
    a, b = blank(20, Hk, page, d, 8), blank(20, Hk, page, d, 8)
    qa, qb = run(a), run(b)
    run(b)  # over again: the same tokens at the same scales
    assert torch.equal(qa, qb) and all(same(x, y) for x, y in zip(a, b))
    both = torch.zeros((20, 2, Hk, page, d), device="cuda").to(torch.float8_e4m3fn)
    c = (both[:, 0], both[:, 1], torch.zeros((20, Hk), device="cuda"), torch.zeros((20, Hk), device="cuda"))
    run(c)
    held = table.view(-1).long()[[b * 4 + j for b in range(B) for j in range(-(-int(lens[b]) // page))]]
    for i in range(2):
        x, y = c[i].contiguous().view(torch.uint8), a[i].view(torch.uint8)
        assert torch.equal(x[held], y[held])
    s = torch.cuda.Stream()
    e = blank(20, Hk, page, d, 8)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qe = q.clone()
        assert run(e, qe, q_out=qe) is qe
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(qe, qa) and all(same(x, y) for x, y in zip(a, e))
    f = blank(20, Hk, page, d, 8)
    qf = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(f, q_out=qf)
    for x in f[:2]:
        x.view(torch.uint8).zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qf, qa) and all(same(x, y) for x, y in zip(a, f))
    # a fused projection's rows [T, H + 2 Hk, d]
    fused = torch.cat((q, k, v)).transpose(0, 1).contiguous().transpose(0, 1)
    h = blank(20, Hk, page, d, 8)
    qh = blk.kv_append_paged(fused[H:H + Hk], fused[H + Hk:], h[0], h[1], table, lens, cu_seqlens=cu, k_scale=h[2],
                             v_scale=h[3], rope=plan, q=fused[:H])
    assert torch.equal(qh, qa) and all(same(x, y) for x, y in zip(a, h))


def test_lengths_and_tables_that_do_not_fit():
    """Tokens with negative positions, and those whose page is not there, take no part; falling
    offsets are clamped: nothing is written outside what the table names."""
    Hk, d, page = 2, 64, 16
    k, v = (randn((Hk, 40, d), "bf16", gen(i)) for i in (1, 2))
    c = blank(6, Hk, page, d, 16)
    # sequence 0: ten of 20 tokens have negative positions; 1: its second page is outside the pool; 2: length 0
    table = i32([[1, 2], [3, 77], [4, -1]])
    blk.kv_append_paged(k, v, *c[:2], table, i32([10, 20, 0]), cu_seqlens=i32([0, 20, 40, 40]))
    assert torch.equal(c[0][1, :, :10], k[:, 10:20]) and torch.equal(c[1][3, :, :16], v[:, 20:36])
    rest = c[0].float()
    rest[1, :, :10] = 0
    rest[3] = 0
    assert not rest.any()
    for cu in ([0, 50, 20, 40], [-7, 10, 5, 1000], [40, 0, 40, 0], [2 ** 31 - 1, -2 ** 31, 3, 9]):
        c = blank(6, Hk, page, d, 8)
        blk.kv_append_paged(k, v, *c[:2], table, i32([32, 2 ** 31 - 1, 31]), cu_seqlens=i32(cu), k_scale=c[2], v_scale=c[3])
        torch.cuda.synchronize()
        for x in c[:2]:
            assert not x.float()[[0, 5]].any()
    blk.check_device_status()


def test_pool_beyond_32_bit_offsets():
    Hk, page, d = 2, 128, 128
    pages = (1 << 32) // (Hk * page * d) + 3
    c = [torch.zeros((pages, Hk, page, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in "kv"]
    s = [torch.zeros((pages, Hk), device="cuda") for _ in "kv"]
    k, v = (randn((Hk, 200, d), "bf16", gen(i)) for i in (3, 4))
    table = i32([[pages - 1, pages - 2], [0, 1]])
    blk.kv_append_paged(k, v, *c, table, i32([200, 0]), cu_seqlens=i32([0, 200, 200]), k_scale=s[0], v_scale=s[1])
    got = (c[1][pages - 1].float() * s[1][pages - 1][:, None, None])
    assert float((got - v[:, :128].float()).abs().max()) <= 2.0 ** -4 * float(v.float().abs().max())
    assert not c[1][:2].view(torch.uint8).any()
    # ... and the decode step over it: keys and values there, by 64-bit offsets
    q = randn((2, 4, d), "bf16", gen(9))
    o = blk.attn_decode_paged(q, *c, table, i32([200, 0]), k_scale=s[0], v_scale=s[1])
    kr, seen, _ = ref.rows(c[0], s[0], [pages - 1, pages - 2], 200, page)
    vr, _, _ = ref.rows(c[1], s[1], [pages - 1, pages - 2], 200, page)
    want, mag, _ = ref.decode(f64(q[0].float()), kr, vr, seen)
    assert (np.abs(f64(o[0].float()) - want) <= 2.0 ** -7 * mag + 2.0 ** -8 * np.abs(want)).all() and not o[1].any()


def test_rope_strides_and_gradient():
    """[T, H, d] transposed, and a slice; the inverse is the gradient of a rotation's call."""
    g = gen(8)
    x = randn((50, 6, 128), "fp16", g)
    pos = torch.randint(-1000, 1000, (50,), generator=g, device="cuda", dtype=torch.int32)  # negative ones too
    plan = blk.rope_plan(64, 10000.0, amplitude=0.75)
    a = blk.rope_positions(x.transpose(0, 1), pos, plan)
    assert torch.equal(a, blk.rope_positions(x.transpose(0, 1).contiguous(), pos, plan))
    q, k = blk.rope_positions(x.transpose(0, 1)[:4], pos, plan, k=x.transpose(0, 1)[4:])
    assert torch.equal(torch.cat((q, k)), a)
    want, mag = ref.turn(f64(x.transpose(0, 1).float()), f64(pos), ref.thetas(64), False, 0.75)
    close(a, want, mag, "fp16")
    # <turn(x), y> = <x, turn back(y)>, each product rounded: u of the terms' magnitudes
    y = randn((6, 50, 128), "fp16", g)
    b = blk.rope_positions(y, pos, plan, inverse=True)
    left, right = (a.double() * y.double()).sum(), (x.transpose(0, 1).double() * b.double()).sum()
    terms = (a.double() * y.double()).abs().sum() + (x.transpose(0, 1).double() * b.double()).abs().sum()
    assert abs(float(left - right)) <= 2.0 ** -10 * float(terms)
    # differences of the turn along y: it is linear, so they are the turn of y
    one = blk.rope_positions((x.transpose(0, 1).double() + y.double()).half(), pos, plan).double()
    two, far = ref.turn(f64((x.transpose(0, 1).double() + y.double()).half()), f64(pos), ref.thetas(64), False, 0.75)
    assert (np.abs(f64(one) - two) <= far * 2.0 ** -20 + 2.0 ** -11 * np.abs(two) * (1 + 2.0 ** -10) + 2.0 ** -25).all()


@pytest.mark.parametrize("d,span", [(256, 256), (160, 40), (256, 250), (160, 0)])
def test_pages_in_rounds(d, span):
    """8-bit pages of more values than a block holds at a time are read twice: whole pages, part-full ones that
    are gone on with, and an infinity in one."""
    for layout in ("heads", "tokens"):
        case(2, 2, d, span, 128, [0, 100, 127, 5], [300, 156, 1, 20], "bf16", 8, seed=d + span, layout=layout,
             with_q=span > 0, loud=2.0)
    k = randn((1, 128, d), "bf16", gen(d)) * 3
    v = k.clone()
    v[0, 77, d - 1] = -float("inf")
    c = blank(2, 1, 128, d, 8)
    blk.kv_append_paged(k, v, *c[:2], i32([[1]]), i32([128]), cu_seqlens=i32([0, 128]), k_scale=c[2], v_scale=c[3])
    fin = v[torch.isfinite(v)].float()
    s = float(c[3][1, 0])
    assert s == ref.page_scale(float(fin.abs().max())) and c[1][1, 0, 77, d - 1].float() == -448
    want = ref.e4m3(np.clip(f64(v[0].float()) / s, -448, 448))
    assert np.array_equal(f64(c[1][1, 0].float()), want)
    assert torch.equal(c[2][1], torch.tensor([ref.page_scale(float(k.float().abs().max()))], device="cuda"))


def test_many_tokens_and_heads():
    """Blocks that take several heads of keys, of values and of queries in turn, the last of each part-filled."""
    for H, Hk, d, span, page, bits in ((40, 10, 64, 32, 16, 8), (23, 23, 64, 64, 32, 8), (40, 10, 128, 128, 64, 8),
                                       (9, 3, 160, 40, 64, 16), (5, 5, 128, 128, 128, 8), (23, 23, 64, 16, 128, 16)):
        case(H, Hk, d, span, page, [0, 33, 0, 700], [1200, 1500, 9, 800], "bf16", bits, interleaved=H == 40, seed=H)
