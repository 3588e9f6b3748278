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
