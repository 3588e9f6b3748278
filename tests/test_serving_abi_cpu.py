"""blk_attn_prefill_packed and blk_attn_decode_shared without a GPU: workspace
sizes and refusals, before any CUDA call."""
import ctypes as C

import pytest

from alibi_attention_block_gb300 import _abi, build

FAKE = 0x100000  # 16-byte-aligned stand-in address; validation rejects before any access
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def desc(tokens=1000, prompts=7, H=32, Hk=8, d=128, prefix=0, scale=-1.0, alibi=0):
    return _abi.PackedDesc(tokens, prompts, H, Hk, d, prefix, scale, alibi)


def call(lib, d, q=FAKE, k=FAKE, v=FAKE, kp=None, vp=None, cu=FAKE, slopes=None, o=FAKE, ws=FAKE,
         n=BIG, dt=1):
    return lib.blk_attn_prefill_packed(C.byref(d), q, k, v, kp, vp, cu, slopes, o, ws, n, dt, None)


@pytest.mark.parametrize("H,Hk,d,alibi,unit", [
    (32, 32, 64, 0, 256), (8, 2, 64, 1, 256), (16, 16, 128, 1, 256), (32, 8, 128, 0, 64),
    (32, 8, 128, 1, 32), (32, 8, 160, 0, 64), (6, 2, 128, 0, 80), (32, 1, 160, 1, 8), (2, 2, 160, 0, 256), (2, 2, 160, 1, 256), (32, 8, 160, 1, 32)])
def test_workspace_size(lib, H, Hk, d, alibi, unit):
    """Nothing up to 256 prompts and 1024 units; above, one 16-byte entry for
    each unit that the prompts can have at most, and one for their count, in
    whole 256 bytes."""
    need = C.c_size_t(0)
    for tokens, prompts in ((1000, 7), (1000, 256), (1000, 257), ((1024 - 3) * unit, 3),
                            ((1024 - 3) * unit, 4), (1 << 20, 5000)):
        units = tokens // unit + prompts
        assert lib.blk_attn_prefill_packed_workspace_size(
            C.byref(desc(tokens, prompts, H, Hk, d, alibi=alibi)), C.byref(need)) == _abi.BLK_OK
        small = prompts <= 256 and units <= 1024
        assert need.value == (0 if small else -(-16 * (1 + units) // 256) * 256)


@pytest.mark.parametrize("bad,status", [
    (dict(tokens=0), _abi.BLK_EINVAL), (dict(tokens=(1 << 30) + 1), _abi.BLK_EINVAL),
    (dict(prompts=0), _abi.BLK_EINVAL), (dict(prompts=(1 << 20) + 1), _abi.BLK_EINVAL),
    (dict(prefix=-1), _abi.BLK_EINVAL), (dict(prefix=(1 << 30) + 1), _abi.BLK_EINVAL),
    (dict(H=30), _abi.BLK_EINVAL), (dict(H=0), _abi.BLK_EINVAL), (dict(Hk=0), _abi.BLK_EINVAL),
    (dict(d=96), _abi.BLK_EUNSUPPORTED), (dict(d=32), _abi.BLK_EUNSUPPORTED),
    (dict(alibi=2), _abi.BLK_EINVAL), (dict(scale=float("nan")), _abi.BLK_EINVAL),
    (dict(tokens=1 << 30, H=4096, Hk=4096, d=64), _abi.BLK_EINVAL),
])
def test_descriptor_refusals(lib, bad, status):
    need = C.c_size_t(0)
    assert lib.blk_attn_prefill_packed_workspace_size(C.byref(desc(**bad)), C.byref(need)) == status
    assert call(lib, desc(**bad), kp=FAKE, vp=FAKE) == status


def test_argument_refusals(lib):
    d = desc()
    assert lib.blk_attn_prefill_packed_workspace_size(C.byref(d), None) == _abi.BLK_EINVAL
    assert lib.blk_attn_prefill_packed_workspace_size(None, None) == _abi.BLK_EINVAL
    for name in ("q", "k", "v", "cu", "o"):
        assert call(lib, d, **{name: None}) == _abi.BLK_EINVAL, name
    for name in ("q", "k", "v", "o"):
        assert call(lib, d, **{name: FAKE + 8}) == _abi.BLK_EINVAL, name
    assert call(lib, d, cu=FAKE + 2) == _abi.BLK_EINVAL
    assert call(lib, d, dt=2) == _abi.BLK_EINVAL
    assert call(lib, d, kp=FAKE) == _abi.BLK_EINVAL          # a prefix of length 0
    p = desc(prefix=5)
    assert call(lib, p, kp=FAKE) == _abi.BLK_EINVAL          # v_prefix missing
    assert call(lib, p, kp=FAKE, vp=FAKE + 4) == _abi.BLK_EINVAL
    assert call(lib, d, slopes=FAKE) == _abi.BLK_EINVAL      # slopes without ALiBi
    assert call(lib, desc(alibi=1), slopes=FAKE + 2) == _abi.BLK_EINVAL
    assert call(lib, desc(H=24, Hk=8, alibi=1)) == _abi.BLK_EUNSUPPORTED
    many = desc(prompts=300)  # a work list in the workspace
    assert call(lib, many, ws=None) == _abi.BLK_EWORKSPACE
    assert call(lib, many, ws=FAKE + 4) == _abi.BLK_EWORKSPACE
    assert call(lib, many, n=64) == _abi.BLK_EWORKSPACE


# ---------------------------------------------- blk_attn_decode_shared --

def shared(batch=4, max_seq=64, H=32, Hk=8, d=128, prefix=1000, scale=-1.0, alibi=0):
    return _abi.DecodeSharedDesc(batch, max_seq, H, Hk, d, prefix, scale, alibi)


def step(lib, d, q=FAKE, kp=FAKE, vp=FAKE, k=FAKE, v=FAKE, lens=FAKE, slopes=None, o=FAKE, ws=FAKE,
         n=BIG, dt=1):
    return lib.blk_attn_decode_shared(C.byref(d), q, kp, vp, k, v, lens, slopes, o, ws, n, dt, None)


@pytest.mark.parametrize("bad,status", [
    (dict(batch=0), _abi.BLK_EINVAL), (dict(max_seq=0), _abi.BLK_EINVAL),
    (dict(prefix=-1), _abi.BLK_EINVAL), (dict(prefix=(1 << 30) + 1), _abi.BLK_EINVAL),
    (dict(H=30), _abi.BLK_EINVAL), (dict(H=24, Hk=8), _abi.BLK_EUNSUPPORTED),
    (dict(d=160), _abi.BLK_EUNSUPPORTED), (dict(d=32), _abi.BLK_EUNSUPPORTED),
    (dict(alibi=3), _abi.BLK_EINVAL), (dict(scale=float("inf")), _abi.BLK_EINVAL),
    (dict(batch=1 << 20, max_seq=1, Hk=32, prefix=1 << 20), _abi.BLK_EINVAL),  # too many tiles
])
def test_shared_descriptor_refusals(lib, bad, status):
    need = C.c_size_t(0)
    assert lib.blk_attn_decode_shared_workspace_size(C.byref(shared(**bad)), C.byref(need)) == status
    assert step(lib, shared(**bad)) == status


def test_shared_argument_refusals(lib):
    d = shared()
    need = C.c_size_t(0)
    assert lib.blk_attn_decode_shared_workspace_size(C.byref(d), C.byref(need)) == _abi.BLK_OK
    assert lib.blk_attn_decode_shared_workspace_size(C.byref(d), None) == _abi.BLK_EINVAL
    for name in ("q", "kp", "vp", "k", "v", "o", "lens"):
        assert step(lib, d, **{name: None}) == _abi.BLK_EINVAL, name
    for name in ("q", "kp", "vp", "k", "v", "o"):
        assert step(lib, d, **{name: FAKE + 8}) == _abi.BLK_EINVAL, name
    assert step(lib, d, lens=FAKE + 1) == _abi.BLK_EINVAL
    assert step(lib, d, dt=7) == _abi.BLK_EINVAL
    assert step(lib, shared(prefix=0)) == _abi.BLK_EINVAL     # a prefix of length 0
    assert step(lib, d, slopes=FAKE) == _abi.BLK_EINVAL       # slopes without ALiBi
    assert step(lib, shared(alibi=1), slopes=FAKE + 2) == _abi.BLK_EINVAL
    assert step(lib, shared(H=48, Hk=12, alibi=1)) == _abi.BLK_EUNSUPPORTED
    assert step(lib, d, ws=None) == _abi.BLK_EWORKSPACE
    assert step(lib, d, ws=FAKE + 8) == _abi.BLK_EWORKSPACE
    assert step(lib, d, n=need.value - 1) == _abi.BLK_EWORKSPACE


@pytest.mark.parametrize("few,many", [
    (dict(prefix=300, max_seq=84), dict(prefix=300, max_seq=85)),                    # 384 keys of 128
    (dict(d=64, Hk=32, prefix=0, max_seq=768, batch=1), dict(d=64, Hk=32, prefix=1, max_seq=768, batch=1)),
    (dict(batch=19, H=16, Hk=16, prefix=20, max_seq=1), dict(batch=20, H=16, Hk=16, prefix=20, max_seq=1)),
    (dict(batch=9, prefix=100, max_seq=99), dict(batch=9, prefix=100, max_seq=100)),  # 288 blocks
])
def test_shared_small_needs_no_workspace(lib, few, many):
    need = C.c_size_t(1)
    size = lib.blk_attn_decode_shared_workspace_size
    assert size(C.byref(shared(**few)), C.byref(need)) == _abi.BLK_OK and need.value == 0
    assert size(C.byref(shared(**many)), C.byref(need)) == _abi.BLK_OK and need.value > 0


# -------------------------------------------------- blk_forward_packed --

def block(batch=1, seq=500, H=4, Hk=4, d=64, span=16):
    q = _abi.QkvDesc(batch, seq, 256, H, Hk, d, _abi.BLK_QKV_STACKED, _abi.BLK_QKNORM_NONE, 1e-5, span, 1e4)
    return _abi.BlockDesc(q, _abi.BLK_NORM_LAYERNORM, _abi.BLK_NORM_PRE, _abi.BLK_RESIDUAL_SEQUENTIAL,
                          1e-5, 0, 688, _abi.BLK_ACT_SWIGLU)


def test_forward_packed_refusals(lib):
    need, dense = C.c_size_t(0), C.c_size_t(0)
    d = block()
    assert lib.blk_forward_workspace_size(C.byref(d), C.byref(dense)) == _abi.BLK_OK
    for prompts, extra in ((3, 0), (300, -(-16 * (1 + 1 + 300) // 256) * 256)):
        assert lib.blk_forward_packed_workspace_size(C.byref(d), prompts, C.byref(need)) == _abi.BLK_OK
        assert need.value == dense.value + extra
    size = lib.blk_forward_packed_workspace_size
    assert size(C.byref(d), 3, None) == _abi.BLK_EINVAL
    assert size(C.byref(d), 0, C.byref(need)) == _abi.BLK_EINVAL
    assert size(C.byref(block(batch=2)), 3, C.byref(need)) == _abi.BLK_EINVAL
    assert size(C.byref(block(d=96)), 3, C.byref(need)) == _abi.BLK_EUNSUPPORTED
    # positions of a rotary are held in 32-bit floats
    assert size(C.byref(block(seq=2**24)), 3, C.byref(need)) == _abi.BLK_OK
    assert size(C.byref(block(seq=2**24 + 1)), 3, C.byref(need)) == _abi.BLK_EINVAL
    assert size(C.byref(block(seq=2**24 + 1, span=0)), 3, C.byref(need)) == _abi.BLK_OK
    w = _abi.BlockWeights(**{n: FAKE for n in ("attn_norm_w", "mlp_norm_w", "w_qkv", "w_o", "w_gate", "w_up",
                                               "w_down")})

    def run(d=d, w=w, cu=FAKE, prompts=3, x=FAKE, y=FAKE * 2, ws=FAKE, n=BIG, dt=1):
        return lib.blk_forward_packed(C.byref(d), C.byref(w), cu, prompts, x, y, ws, n, dt, None)

    assert run(cu=None) == _abi.BLK_EINVAL
    assert run(cu=FAKE + 2) == _abi.BLK_EINVAL
    assert run(prompts=0) == _abi.BLK_EINVAL
    assert run(d=block(batch=2)) == _abi.BLK_EINVAL
    assert run(w=_abi.BlockWeights()) == _abi.BLK_EINVAL
    assert run(x=None) == _abi.BLK_EINVAL
    assert run(y=FAKE) == _abi.BLK_EINVAL                      # y aliases x
    assert run(dt=5) == _abi.BLK_EINVAL
    assert run(n=dense.value - 1) == _abi.BLK_EWORKSPACE
    assert run(ws=None) == _abi.BLK_EWORKSPACE
