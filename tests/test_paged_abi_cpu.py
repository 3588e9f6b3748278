"""The paged cache's calls and the rotary's plan without a GPU: the plan's numbers, workspace
sizes, and refusals before any CUDA call, of the C calls and of the binding."""
import ctypes as C
import math
from fractions import Fraction

import pytest
import torch

import alibi_attention_block_gb300 as blk
from alibi_attention_block_gb300 import _abi, build

FAKE = 0x100000  # 16-byte-aligned stand-in address; validation rejects before any access
BIG = 1 << 40
EINVAL, EUNSUPPORTED, EWORKSPACE = _abi.BLK_EINVAL, _abi.BLK_EUNSUPPORTED, _abi.BLK_EWORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


# ------------------------------------------------------------------ plan --
@pytest.mark.parametrize("span,base,more", [
    (128, 10000.0, {}), (40, 500000.0, {}), (2, 1.0, {}), (256, 10000.0, dict(scaling="linear", factor=8.0)),
    (64, 10000.0, dict(scaling="by_parts", factor=16.0, original_len=4096.0, beta_slow=1.0, beta_fast=32.0))])
def test_plan_angles(lib, span, base, more):
    """turns: the angle per position in 2^-64 turns, off by the 53 bits of theta's arithmetic (a few
    roundings, each 2^-53)."""
    plan = blk.rope_plan(span, base, interleaved=span == 40, amplitude=1.5, **more)
    assert (plan.pairs, plan.interleaved, plan.amplitude) == (span // 2, int(span == 40), 1.5)
    for j in range(span // 2):
        th = base ** (-2.0 * j / span)
        f = more.get("factor", 1.0)
        if more.get("scaling") == "linear":
            th /= f
        elif more.get("scaling") == "by_parts":
            g = min(1.0, max(0.0, (more["original_len"] * th / (2 * math.pi) - 1.0) / 31.0))
            th = g * th + (1 - g) * th / f
        turns = Fraction(th) / Fraction(2 * math.pi)
        assert abs(Fraction(plan.turns[j], 2 ** 64) - turns) <= turns / 2 ** 49 + Fraction(1, 2 ** 64)
    assert not any(plan.turns[j] for j in range(span // 2, 128))


@pytest.mark.parametrize("bad", [
    dict(span=0), dict(span=3), dict(span=258), dict(span=-2), dict(base=0.5), dict(base=float("nan")),
    dict(base=float("inf")), dict(amplitude=0.0), dict(amplitude=-1.0), dict(amplitude=float("nan")),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("inf")),
    dict(scaling="by_parts", factor=2.0), dict(scaling="by_parts", factor=2.0, original_len=100, beta_slow=32.0),
])
def test_plan_refusals(lib, bad):
    with pytest.raises(blk.BlkError):
        blk.rope_plan(**{"span": 64, **bad})


def test_plan_refusals_of_the_library(lib):
    d, p = _abi.RopeDesc(64, 0, 1e4, 0, 1.0, 1.0, 0, 1, 32), _abi.RopePlan()
    assert lib.blk_rope_plan_init(C.byref(d), C.byref(p)) == _abi.BLK_OK
    assert lib.blk_rope_plan_init(None, C.byref(p)) == EINVAL
    assert lib.blk_rope_plan_init(C.byref(d), None) == EINVAL
    for field, value in (("scaling", 3), ("scaling", -1), ("interleaved", 2)):
        e = _abi.RopeDesc.from_buffer_copy(d)
        setattr(e, field, value)
        assert lib.blk_rope_plan_init(C.byref(e), C.byref(p)) == EINVAL
    with pytest.raises(ValueError):
        blk.rope_plan(64, scaling="other")


# ------------------------------------------------------------- positions --
def rope(lib, plan="made", q=FAKE, k=FAKE, pos=FAKE, qo=FAKE * 2, ko=FAKE * 3, dt=1, **kw):
    f = dict(tokens=10, n_heads=4, n_k_heads=2, head_dim=128, inverse=0, q_head_stride=1280, q_token_stride=128,
             q_out_head_stride=1280, q_out_token_stride=128, k_head_stride=1280, k_token_stride=128,
             k_out_head_stride=1280, k_out_token_stride=128)
    f.update(kw)
    p = blk.rope_plan(128) if plan == "made" else plan
    return lib.blk_rope_positions(C.byref(_abi.RopePosDesc(**f)), None if p is None else C.byref(p), q, k, pos, qo,
                                  ko, dt, None)


@pytest.mark.parametrize("bad", [
    dict(tokens=0), dict(tokens=(1 << 30) + 1), dict(n_heads=0), dict(n_heads=1 << 15), dict(head_dim=120),
    dict(head_dim=272), dict(head_dim=64), dict(inverse=2), dict(n_k_heads=0), dict(n_k_heads=-1), dict(k=None),
    dict(ko=None), dict(q=None), dict(qo=None), dict(pos=None), dict(pos=FAKE + 2), dict(q=FAKE + 8),
    dict(ko=FAKE + 8), dict(q_head_stride=4), dict(k_token_stride=-8), dict(q_out_token_stride=1 << 41), dict(dt=2),
    dict(plan=None), dict(plan=_abi.RopePlan()), dict(qo=FAKE, q_out_head_stride=2560)])
def test_rope_refusals(lib, bad):
    assert rope(lib, **bad) == EINVAL


# ---------------------------------------------------------------- cache --
def cache(pages=9, page=16, Hk=2, d=128, B=3, max_pages=40, stride=None, kind=1):
    return _abi.PagedDesc(pages, page, Hk, d, B, max_pages, Hk * page * d if stride is None else stride, kind)


BAD_CACHES = [
    (dict(pages=0), EINVAL), (dict(pages=(1 << 30) + 1), EINVAL), (dict(page=24), EUNSUPPORTED),
    (dict(page=8), EUNSUPPORTED), (dict(page=256), EUNSUPPORTED), (dict(Hk=0), EINVAL), (dict(Hk=5000), EINVAL),
    (dict(d=136), EUNSUPPORTED), (dict(d=0), EUNSUPPORTED), (dict(d=272), EUNSUPPORTED), (dict(B=0), EINVAL),
    (dict(B=(1 << 24) + 1), EINVAL), (dict(max_pages=0), EINVAL), (dict(max_pages=1 << 28), EINVAL),
    (dict(max_pages=(1 << 22) + 1), EINVAL),
    (dict(stride=2 * 16 * 128 - 16), EINVAL), (dict(stride=2 * 16 * 128 + 8), EINVAL), (dict(stride=1 << 40), EINVAL),
    (dict(pages=1 << 30, stride=1 << 30), EINVAL), (dict(kind=2), EINVAL), (dict(kind=-1), EINVAL)]


def append(lib, c=None, plan=None, k=FAKE, v=FAKE, q=None, cu=FAKE, pos=None, table=FAKE, lens=FAKE, kc=FAKE, vc=FAKE,
           ks=FAKE, vs=FAKE, qo=None, dt=1, **kw):
    f = dict(tokens=10, n_heads=0, k_head_stride=1280, k_token_stride=128, v_head_stride=1280, v_token_stride=128,
             q_head_stride=1280, q_token_stride=128, q_out_head_stride=1280, q_out_token_stride=128)
    f.update(kw)
    d = _abi.AppendDesc(cache=cache() if c is None else c, **f)
    return lib.blk_kv_append_paged(C.byref(d), None if plan is None else C.byref(plan), k, v, q, cu, pos, table, lens,
                                   kc, vc, ks, vs, qo, dt, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_cache_refusals(lib, bad, status):
    need = C.c_size_t(0)
    assert append(lib, cache(**bad)) == status
    d = _abi.DecodePagedDesc(cache(**bad), 4, 512, 128, -1.0, 0)
    assert lib.blk_attn_decode_paged_workspace_size(C.byref(d), C.byref(need)) == status
    assert step(lib, cache(**bad)) == status


@pytest.mark.parametrize("bad", [
    dict(tokens=0), dict(tokens=(1 << 30) + 1), dict(cu=None), dict(cu=FAKE + 1), dict(k=None), dict(v=None),
    dict(k=FAKE + 4), dict(table=None), dict(table=FAKE + 2), dict(lens=None), dict(kc=None), dict(vc=FAKE + 8),
    dict(ks=None), dict(vs=FAKE + 2), dict(n_heads=4), dict(q=FAKE), dict(q=FAKE, qo=FAKE), dict(n_heads=4, q=FAKE),
    dict(n_heads=20000, q=FAKE, qo=FAKE), dict(pos=FAKE), dict(plan=_abi.RopePlan()), dict(k_head_stride=12),
    dict(v_token_stride=-8),
    dict(k_token_stride=1 << 24), dict(n_heads=4, q=FAKE, qo=FAKE, q_head_stride=64), dict(dt=3)])
def test_append_refusals(lib, bad):
    assert append(lib, **bad) == EINVAL


def test_append_more_refusals(lib):
    assert append(lib, cache(kind=0)) == EINVAL                       # scales of a 16-bit cache
    assert append(lib, plan=blk.rope_plan(160)) == EINVAL             # a span above head_dim
    assert append(lib, plan=blk.rope_plan(128), pos=FAKE + 2) == EINVAL
    assert lib.blk_kv_append_paged(None, None, FAKE, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None,
                                   1, None) == EINVAL


def step(lib, c=None, H=4, qb=512, qh=128, scale=-1.0, alibi=0, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE,
         lens=FAKE, slopes=None, o=FAKE, ws=FAKE, n=BIG, dt=1):
    d = _abi.DecodePagedDesc(cache() if c is None else c, H, qb, qh, scale, alibi)
    return lib.blk_attn_decode_paged(C.byref(d), q, kc, vc, ks, vs, table, lens, slopes, o, ws, n, dt, None)


@pytest.mark.parametrize("bad,status", [
    (dict(H=0), EINVAL), (dict(H=3), EINVAL), (dict(H=1 << 15), EINVAL), (dict(qb=-2), EINVAL), (dict(qh=3), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(alibi=2), EINVAL), (dict(c=cache(d=96)), EUNSUPPORTED),
    (dict(c=cache(d=256)), EUNSUPPORTED), (dict(q=None), EINVAL), (dict(o=FAKE + 8), EINVAL), (dict(kc=None), EINVAL),
    (dict(vs=None), EINVAL), (dict(table=None), EINVAL), (dict(lens=FAKE + 1), EINVAL), (dict(slopes=FAKE), EINVAL),
    (dict(slopes=FAKE + 2, alibi=1), EINVAL), (dict(H=6, alibi=1), EUNSUPPORTED), (dict(dt=9), EINVAL),
    (dict(ws=None), EWORKSPACE), (dict(ws=FAKE + 8), EWORKSPACE), (dict(n=1000), EWORKSPACE),
    (dict(c=cache(B=1 << 24), H=64), EINVAL)])
def test_decode_refusals(lib, bad, status):
    assert step(lib, **bad) == status


def test_workspace(lib):
    """Room for a record per CTA and per unit; none where sequences have four tiles of 128 keys at most."""
    def need(**kw):
        n = C.c_size_t(1)
        d = _abi.DecodePagedDesc(cache(**kw), 16, 2048, 128, -1.0, 0)
        assert lib.blk_attn_decode_paged_workspace_size(C.byref(d), C.byref(n)) == _abi.BLK_OK
        return n.value
    assert need(max_pages=32) == 0 and need(page=128, max_pages=4) == 0
    assert need(max_pages=33) >= (640 + 3 * 2) * 8 * (128 + 2) * 4
    d = _abi.DecodePagedDesc(cache(), 16, 2048, 128, -1.0, 0)
    assert lib.blk_attn_decode_paged_workspace_size(C.byref(d), None) == EINVAL
    assert lib.blk_attn_decode_paged_workspace_size(None, C.byref(C.c_size_t())) == EINVAL


# -------------------------------------------------------------- binding --
def tensors():
    z, i = torch.zeros, torch.int32
    f8 = torch.float8_e4m3fn
    return dict(k=z(2, 5, 64, dtype=torch.bfloat16), v=z(2, 5, 64, dtype=torch.bfloat16),
                k_cache=z(7, 2, 16, 64, dtype=f8), v_cache=z(7, 2, 16, 64, dtype=f8), block_table=z(3, 4, dtype=i),
                lens=z(3, dtype=i), cu_seqlens=z(4, dtype=i), k_scale=z(7, 2), v_scale=z(7, 2))


@pytest.mark.parametrize("name,value,error", [
    ("k", torch.zeros(2, 5, 64), TypeError), ("v", torch.zeros(2, 4, 64, dtype=torch.bfloat16), ValueError),
    ("v", torch.zeros(2, 5, 64, dtype=torch.float16), TypeError),
    ("k", torch.zeros(2, 64, 5, dtype=torch.bfloat16).transpose(1, 2), ValueError),
    ("k_cache", torch.zeros(7, 2, 16, 64, dtype=torch.float16), TypeError),
    ("k_cache", torch.zeros(7, 2, 16, 64, dtype=torch.bfloat16), ValueError),
    ("v_cache", torch.zeros(6, 2, 16, 64, dtype=torch.float8_e4m3fn), ValueError),
    ("v_cache", torch.zeros(14, 2, 16, 64, dtype=torch.float8_e4m3fn)[::2], ValueError),
    ("k_cache", torch.zeros(7, 16, 2, 64, dtype=torch.float8_e4m3fn).transpose(1, 2), ValueError),
    ("k_scale", None, ValueError), ("v_scale", torch.zeros(7, 3), ValueError),
    ("k_scale", torch.zeros(7, 2, dtype=torch.float16), TypeError), ("k_scale", torch.zeros(2, 7).t(), ValueError),
    ("block_table", torch.zeros(3, 4, dtype=torch.int64), TypeError), ("lens", torch.zeros(4, dtype=torch.int32), ValueError),
    ("block_table", torch.zeros(3, 8, dtype=torch.int32)[:, ::2], ValueError),
    ("cu_seqlens", torch.zeros(3, dtype=torch.int32), ValueError), ("lens", [1, 2, 3], TypeError),
    ("q", torch.zeros(4, 6, 64, dtype=torch.bfloat16), ValueError), ("q_out", torch.zeros(4, 5, 64), ValueError),
    ("positions", torch.zeros(6, dtype=torch.int32), ValueError)])
def test_binding_append_refusals(lib, name, value, error):
    with pytest.raises(error):
        blk.kv_append_paged(**{**tensors(), name: value})


@pytest.mark.parametrize("name,value,error", [
    ("q", torch.zeros(3, 4, 64), TypeError), ("q", torch.zeros(2, 4, 64, dtype=torch.bfloat16), ValueError),
    ("q", torch.zeros(3, 4, 128, dtype=torch.bfloat16), ValueError), ("q", torch.zeros(4, 64, dtype=torch.bfloat16), ValueError),
    ("out", torch.zeros(3, 4, 64), TypeError), ("out", torch.zeros(4, 3, 64, dtype=torch.bfloat16).transpose(0, 1), ValueError),
    ("slopes", torch.zeros(3), ValueError), ("k_scale", None, ValueError),
    ("q", torch.zeros(3, 3, 64, dtype=torch.bfloat16), blk.BlkError)])
def test_binding_decode_refusals(lib, name, value, error):
    t = tensors()
    for n in ("k", "v", "cu_seqlens"):
        t.pop(n)
    with pytest.raises(error):
        blk.attn_decode_paged(**{"q": torch.zeros(3, 4, 64, dtype=torch.bfloat16), **t, name: value})


def test_binding_rope_refusals(lib):
    q, pos, plan = torch.zeros(4, 5, 64, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32), blk.rope_plan(64)
    for bad, error in ((dict(q=q.float()), TypeError), (dict(positions=pos.long()), TypeError),
                       (dict(positions=pos[:4]), ValueError), (dict(k=q[:, :4]), ValueError),
                       (dict(k=q.half()), TypeError), (dict(k_out=q), ValueError), (dict(q_out=q[:3]), ValueError),
                       (dict(q=q[0]), ValueError), (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                       (dict(positions=[1] * 5), TypeError), (dict(plan=None), TypeError), (dict(plan=64), TypeError)):
        with pytest.raises(error):
            blk.rope_positions(**{"q": q, "positions": pos, "plan": plan, **bad})
