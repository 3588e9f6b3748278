"""GB300 (sm_103a) prefill forward of one decoder block.

A thin torch-facing binding over the C ABI in ``include/blk.h``
(``lib/libblk.so``): it checks tensors, passes device pointers and the current
CUDA stream, and raises ``BlkError`` on a non-OK status. Every step of the
block runs in the library's CUDA kernels; nothing here computes.

Block variants (nnterp encyclopedia "stablelm", 03 Notes; "OLMo-2: reordered
(post) normalization", section 1; "Bloom in a sovereign engine",
Contribution): sequential pre-norm, parallel residual, reordered post-norm;
LayerNorm-with-bias or RMSNorm; stacked or head-interleaved QKV with bias;
full-width or per-head qk-norm; partial NeoX rotary or ALiBi.
"""
from __future__ import annotations

import ctypes as C
import functools

import torch

from . import _abi
from ._abi import BlkError  # noqa: F401

__all__ = ["layernorm_bias", "rmsnorm", "qkv_bias_rope_partial", "rope_inplace", "attn_prefill",
           "attn_prefill_packed", "attn_prefill_packed_workspace_size", "packed_desc",
           "attn_decode", "attn_decode_workspace_size", "decode_desc",
           "attn_decode_shared", "attn_decode_shared_workspace_size", "decode_shared_desc",
           "rope_plan", "rope_positions", "kv_append_paged", "attn_decode_paged",
           "attn_decode_paged_workspace_size", "decode_paged_desc",
           "linear", "mlp", "block_desc", "forward_workspace_size", "forward_q8_0_workspace_size", "forward", "forward_packed", "forward_packed_workspace_size", "forward_host", "ForwardGraph", "HostPipe", "model_desc",
           "model_workspace_size", "model_forward",
           "check_device_status", "BlkError", "library_path"]

library_path = _abi.LIB_PATH


def _lib():
    return _abi.load()


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return _abi.BLK_F16
    if t.dtype == torch.bfloat16:
        return _abi.BLK_BF16
    raise TypeError(f"storage dtype must be float16 or bfloat16, got {t.dtype}")


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensors passed to the block library must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the block library must be contiguous")
    return t.data_ptr()


def _same(dt_tensor, *ts):
    for t in ts:
        if t is not None and t.dtype != dt_tensor.dtype:
            raise TypeError(f"all tensors must share dtype {dt_tensor.dtype}, got {t.dtype}")


def _stream():
    return C.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def layernorm_bias(x, gamma, beta=None, residual=None, eps=1e-5, out=None):
    """y = LN(x) * gamma + beta [+ residual] over the last axis."""
    _same(x, gamma, beta, residual, out)
    out = torch.empty_like(x) if out is None else out
    cols = x.shape[-1]
    _abi.check(_lib().blk_layernorm_bias(_p(x), _p(residual), _p(gamma), _p(beta), _p(out),
                                         x.numel() // cols, cols, eps, _dt(x), _stream()),
               "blk_layernorm_bias")
    return out


def rmsnorm(x, weight, residual=None, eps=1e-6, out=None):
    """y = x / rms(x) * weight [+ residual] over the last axis."""
    _same(x, weight, residual, out)
    out = torch.empty_like(x) if out is None else out
    cols = x.shape[-1]
    _abi.check(_lib().blk_rmsnorm(_p(x), _p(residual), _p(weight), _p(out), x.numel() // cols,
                                  cols, eps, _dt(x), _stream()), "blk_rmsnorm")
    return out


_LAYOUT = {"stacked": _abi.BLK_QKV_STACKED, "head_interleaved": _abi.BLK_QKV_HEAD_INTERLEAVED}
_QKN = {"none": _abi.BLK_QKNORM_NONE, "rms_full": _abi.BLK_QKNORM_RMS_FULL,
        "ln_per_head": _abi.BLK_QKNORM_LN_PER_HEAD}


def _qkv_desc(batch, seq, hidden, n_heads, n_kv_heads, head_dim, layout, qk_norm, qk_norm_eps,
              rotary_span, rope_base):
    return _abi.QkvDesc(batch, seq, hidden, n_heads, n_kv_heads, head_dim, _LAYOUT[layout],
                        _QKN[qk_norm], qk_norm_eps, rotary_span, rope_base)


def qkv_bias_rope_partial(x, w_qkv, b_qkv=None, *, n_heads, n_kv_heads, head_dim,
                          layout="stacked", qk_norm="none", qk_norm_eps=1e-5, rotary_span=0,
                          rope_base=10000.0, q_norm_w=None, k_norm_w=None):
    """x [B, S, D] -> head-split q [B, H, S, d], k and v [B, Hk, S, d]."""
    _same(x, w_qkv, b_qkv, q_norm_w, k_norm_w)
    B, S, D = x.shape
    desc = _qkv_desc(B, S, D, n_heads, n_kv_heads, head_dim, layout, qk_norm, qk_norm_eps,
                     rotary_span, rope_base)
    q = torch.empty((B, n_heads, S, head_dim), dtype=x.dtype, device=x.device)
    k = torch.empty((B, n_kv_heads, S, head_dim), dtype=x.dtype, device=x.device)
    v = torch.empty_like(k)
    _abi.check(_lib().blk_qkv_bias_rope_partial(C.byref(desc), _p(x), _p(w_qkv), _p(b_qkv),
                                                _p(q_norm_w), _p(k_norm_w), _p(q), _p(k), _p(v),
                                                _dt(x), _stream()), "blk_qkv_bias_rope_partial")
    return q, k, v


def rope_inplace(x, bias=None, rotary_span=0, rope_base=10000.0):
    """In place on x [B, n, S, d]: x += bias (per head), then partial NeoX rotary."""
    _same(x, bias)
    B, n, S, d = x.shape
    _abi.check(_lib().blk_rope_inplace(_p(x), _p(bias), B, n, S, d, rotary_span, rope_base,
                                       _dt(x), _stream()), "blk_rope_inplace")
    return x


def attn_prefill(q, k, v, alibi=False, slopes=None, scale=None, out=None):
    """Causal attention: q [B, H, S, d], k/v [B, Hk, S, d] -> o [B, S, H, d]."""
    _same(q, k, v, out)
    B, H, S, d = q.shape
    Hk = k.shape[1]
    if slopes is not None and slopes.dtype != torch.float32:
        raise TypeError("ALiBi slopes are fp32")
    desc = _abi.AttnDesc(B, S, H, Hk, d, -1.0 if scale is None else scale, 1, 1 if alibi else 0)
    o = torch.empty((B, S, H, d), dtype=q.dtype, device=q.device) if out is None else out
    _abi.check(_lib().blk_attn_prefill(C.byref(desc), _p(q), _p(k), _p(v), _p(slopes), _p(o),
                                       _dt(q), _stream()), "blk_attn_prefill")
    return o


def _pointers(dtype, dev, *ts):
    """Device pointers of contiguous tensors of one type on device dev (None
    stays None): _same and _p for a call's tensors in one pass (these calls
    can be shorter than a dozen separate checks)."""
    out = []
    try:
        for t in ts:
            if t is None:
                out.append(None)
            elif t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
                out.append(t.data_ptr())
            else:
                _refuse(t, dtype, dev)
    except AttributeError:
        raise TypeError("expected a torch.Tensor") from None
    return out


def _workspace(t, dev):
    return _pointers(t.dtype, dev, t)[0], t.nbytes


def _with_workspace(call, workspace, need, dev):
    """call(pointer, bytes, stream) on the current stream of device dev, with
    the caller's workspace, or one of `need` bytes from torch's allocator that
    goes back as the call returns, to be used again in the stream's order (as a
    tensor would be, in half its time)."""
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if workspace is not None:
        return call(*_workspace(workspace, dev), stream)
    if not need:
        return call(None, 0, stream)
    ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(need, stream)
    try:
        return call(ptr, need, stream)
    finally:
        torch._C._cuda_cudaCachingAllocator_raw_delete(ptr)


def _refuse(t, dtype, dev):
    if t.dtype is not dtype:
        raise TypeError(f"expected a {dtype} tensor, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("tensors passed to the block library must be CUDA tensors")
    if t.get_device() != dev:
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")
    raise ValueError("tensors passed to the block library must be contiguous")


def _shape(t, want, what):
    if t is not None and t.shape != want:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {want}")


def packed_desc(tokens, prompts, n_heads, n_kv_heads, head_dim, prefix_len=0, alibi=False,
                scale=None):
    return _abi.PackedDesc(tokens, prompts, n_heads, n_kv_heads, head_dim, prefix_len,
                           -1.0 if scale is None else scale, 1 if alibi else 0)


def attn_prefill_packed_workspace_size(desc) -> int:
    need = C.c_size_t(0)
    _abi.check(_lib().blk_attn_prefill_packed_workspace_size(C.byref(desc), C.byref(need)),
               "blk_attn_prefill_packed_workspace_size")
    return need.value


def _values(alibi, scale):
    """A call's switch and scale as plain values: a plan is kept by them, and a
    0-dim tensor given for one hashes by identity, whatever it holds by now."""
    return bool(alibi), None if scale is None else float(scale)


@functools.lru_cache(maxsize=256)
def _packed_plan(*args):
    """(descriptor by reference, workspace bytes) of a call's sizes and _values."""
    desc = packed_desc(*args)
    return C.byref(desc), attn_prefill_packed_workspace_size(desc)


def _prefix_len(k_prefix, v_prefix, n_kv_heads, head_dim):
    if (k_prefix is None) != (v_prefix is None):
        raise ValueError("k_prefix and v_prefix go together")
    if k_prefix is None:
        return 0
    P = k_prefix.shape[1]
    _shape(k_prefix, (n_kv_heads, P, head_dim), "k_prefix")
    _shape(v_prefix, (n_kv_heads, P, head_dim), "v_prefix")
    return P


def attn_prefill_packed(q, k, v, cu_seqlens, k_prefix=None, v_prefix=None, alibi=False,
                        slopes=None, scale=None, out=None, workspace=None):
    """Causal attention over packed prompts: q [H, T, d], k/v [Hk, T, d] hold
    the prompts one behind the other, prompt i in rows cu_seqlens[i] ..
    cu_seqlens[i+1] - 1 (int32 [prompts + 1] on the device). k_prefix /
    v_prefix [Hk, P, d]: keys that every prompt sees ahead of its own. Returns
    o [T, H, d]; rows outside every prompt are not written (pass ``out`` to
    say what they hold)."""
    dt = _dt(q)
    H, T, d = q.shape
    Hk = k.shape[0]
    _shape(k, (Hk, T, d), "k")
    _shape(v, (Hk, T, d), "v")
    P = _prefix_len(k_prefix, v_prefix, Hk, d)
    if P == 0:
        k_prefix = v_prefix = None
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens has shape [prompts + 1]")
    _shape(slopes, (H,), "slopes")
    _shape(out, (T, H, d), "out")
    desc, need = _packed_plan(T, cu_seqlens.numel() - 1, H, Hk, d, P, *_values(alibi, scale))
    dev = torch.cuda.current_device()
    qp, kp, vp, kpp, vpp, op = _pointers(q.dtype, dev, q, k, v, k_prefix, v_prefix, out)
    (cup,) = _pointers(torch.int32, dev, cu_seqlens)
    sp = None if slopes is None else _pointers(torch.float32, dev, slopes)[0]
    o = out
    if o is None:
        o = torch.empty((T, H, d), dtype=q.dtype, device=q.device)
        op = o.data_ptr()
    fn = _lib().blk_attn_prefill_packed
    _abi.check(_with_workspace(
        lambda wp, wn, st: fn(desc, qp, kp, vp, kpp, vpp, cup, sp, op, wp, wn, dt, st),
        workspace, need, dev), "blk_attn_prefill_packed")
    return o


def decode_desc(batch, max_seq, n_heads, n_kv_heads, head_dim, alibi=False, scale=None):
    return _abi.DecodeDesc(batch, max_seq, n_heads, n_kv_heads, head_dim,
                           -1.0 if scale is None else scale, 1 if alibi else 0)


def attn_decode_workspace_size(desc) -> int:
    need = C.c_size_t(0)
    _abi.check(_lib().blk_attn_decode_workspace_size(C.byref(desc), C.byref(need)),
               "blk_attn_decode_workspace_size")
    return need.value


def attn_decode(q, k_cache, v_cache, lens, alibi=False, slopes=None, scale=None, out=None,
                workspace=None):
    """One decode step: q [B, H, d] (newest token of each sequence, at position
    lens[b] - 1) against k/v caches [B, Hk, S_max, d]; lens int32 [B] on the
    device. Returns o [B, H, d]."""
    _same(q, k_cache, v_cache, out)
    B, H, d = q.shape
    Hk, S_max = k_cache.shape[1], k_cache.shape[2]
    if lens.dtype != torch.int32:
        raise TypeError("lens are int32")
    if slopes is not None and slopes.dtype != torch.float32:
        raise TypeError("ALiBi slopes are fp32")
    desc = decode_desc(B, S_max, H, Hk, d, alibi, scale)
    if workspace is None:
        workspace = torch.empty(attn_decode_workspace_size(desc), dtype=torch.uint8,
                                device=q.device)
    o = torch.empty_like(q) if out is None else out
    _abi.check(_lib().blk_attn_decode(C.byref(desc), _p(q), _p(k_cache), _p(v_cache), _p(lens),
                                      _p(slopes), _p(o), _p(workspace), workspace.numel(), _dt(q),
                                      _stream()), "blk_attn_decode")
    return o


def decode_shared_desc(batch, max_seq, n_heads, n_kv_heads, head_dim, prefix_len, alibi=False,
                       scale=None):
    return _abi.DecodeSharedDesc(batch, max_seq, n_heads, n_kv_heads, head_dim, prefix_len,
                                 -1.0 if scale is None else scale, 1 if alibi else 0)


def attn_decode_shared_workspace_size(desc) -> int:
    need = C.c_size_t(0)
    _abi.check(_lib().blk_attn_decode_shared_workspace_size(C.byref(desc), C.byref(need)),
               "blk_attn_decode_shared_workspace_size")
    return need.value


@functools.lru_cache(maxsize=256)
def _decode_shared_plan(*args):
    """(descriptor by reference, workspace bytes) of a call's sizes and _values."""
    desc = decode_shared_desc(*args)
    return C.byref(desc), attn_decode_shared_workspace_size(desc)


def attn_decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, lens, alibi=False, slopes=None,
                       scale=None, out=None, workspace=None):
    """One decode step of a batch that shares a prefix: q [B, H, d] (newest
    token of each sequence, at position P + lens[b] - 1) against k/v_prefix
    [Hk, P, d] (None: no prefix), stored once, and each sequence's own caches
    [B, Hk, S_max, d] of lens[b] keys (int32 [B] on the device, clamped to
    [0, S_max]; 0: the sequence takes no part, its row is zero). Returns o
    [B, H, d]; the softmax weights are rounded to q's type where a workspace is
    needed, and held in 32 bits below (``attn_decode`` always does)."""
    dt = _dt(q)
    B, H, d = q.shape
    Hk, S_max = k_cache.shape[1], k_cache.shape[2]
    _shape(k_cache, (B, Hk, S_max, d), "k_cache")
    _shape(v_cache, (B, Hk, S_max, d), "v_cache")
    P = _prefix_len(k_prefix, v_prefix, Hk, d)
    if P == 0:
        k_prefix = v_prefix = None
    _shape(lens, (B,), "lens")
    _shape(slopes, (H,), "slopes")
    _shape(out, (B, H, d), "out")
    desc, need = _decode_shared_plan(B, S_max, H, Hk, d, P, *_values(alibi, scale))
    dev = torch.cuda.current_device()
    qp, kpp, vpp, kp, vp, op = _pointers(q.dtype, dev, q, k_prefix, v_prefix, k_cache, v_cache, out)
    (lp,) = _pointers(torch.int32, dev, lens)
    sp = None if slopes is None else _pointers(torch.float32, dev, slopes)[0]
    o = out
    if o is None:
        o = torch.empty_like(q)
        op = o.data_ptr()
    fn = _lib().blk_attn_decode_shared
    _abi.check(_with_workspace(
        lambda wp, wn, st: fn(desc, qp, kpp, vpp, kp, vp, lp, sp, op, wp, wn, dt, st),
        workspace, need, dev), "blk_attn_decode_shared")
    return o


_SCALING = {"none": _abi.BLK_ROPE_PLAIN, "linear": _abi.BLK_ROPE_LINEAR,
            "by_parts": _abi.BLK_ROPE_BY_PARTS}


def rope_plan(span, base=10000.0, interleaved=False, scaling="none", factor=1.0, original_len=0.0,
              beta_slow=1.0, beta_fast=32.0, amplitude=1.0):
    """The plan of a rotary for ``rope_positions`` and ``kv_append_paged``, made
    once: span dims of a head, in halves or interleaved pairs, with positions
    scaled "linear" or "by_parts" (blk_rope_scaling in include/blk.h says
    how; the parts are weighted by a pair's turns, not by its index), turned
    dims times amplitude. Plain host data, not to be changed: calls
    with the same values share it."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling must be one of {sorted(_SCALING)}")
    if not -2 ** 31 <= span < 2 ** 31 or span != int(span):
        raise ValueError(f"span must be a whole number of 32 bits, got {span}")
    return _rope_plan(int(span), 1 if interleaved else 0, float(base), _SCALING[scaling], float(amplitude),
                      float(factor), float(original_len), float(beta_slow), float(beta_fast))


@functools.lru_cache(maxsize=64)
def _rope_plan(*fields):
    plan = _abi.RopePlan()
    desc = _abi.RopeDesc(*fields)
    _abi.check(_lib().blk_rope_plan_init(C.byref(desc), C.byref(plan)), "blk_rope_plan_init")
    plan.ref = C.byref(plan)
    return plan


def _plan_ref(plan):
    try:
        return plan.ref
    except AttributeError:
        raise TypeError("a rotary is given as a rope_plan") from None


def _sig(*ts):
    """What a plan is kept by of a call's tensors: type, shape and strides."""
    try:
        return tuple([t if t is None else (t.dtype, t.shape, t.stride()) for t in ts])
    except AttributeError:
        raise TypeError("expected a torch.Tensor") from None


def _addresses(dev, *ts):
    """Device pointers of tensors on device dev (None stays None)."""
    out = []
    for t in ts:
        if t is None:
            out.append(None)
        elif t.get_device() == dev:
            out.append(t.data_ptr())
        else:
            _refuse(t, t.dtype, dev)
    return out


_DT = {torch.float16: _abi.BLK_F16, torch.bfloat16: _abi.BLK_BF16}


def _storage(dtype):
    if dtype not in _DT:
        raise TypeError(f"storage dtype must be float16 or bfloat16, got {dtype}")
    return _DT[dtype]


def _want(sig, dtype, shape, what):
    """A tensor of this type and shape, its axes one behind the other (None: no tensor)."""
    if sig is None:
        return
    if sig[0] is not dtype:
        raise TypeError(f"{what}: expected a {dtype} tensor, got {sig[0]}")
    if sig[1] != shape:
        raise ValueError(f"{what} has shape {tuple(sig[1])}, expected {shape}")
    _dense(sig, what)


def _dense(sig, what):
    n = 1
    for size, stride in zip(reversed(sig[1]), reversed(sig[2])):
        if size != 1 and stride != n:
            raise ValueError(f"{what} must be contiguous")
        n *= size


def _heads(sig, dtype, shape, what):
    """(stride of the first axis, of the second) of a tensor [a, b, dim] with
    contiguous dims. The stride of an axis of length 1 is never used, whatever
    it is."""
    if sig is None:
        return 0, 0
    if sig[0] is not dtype:
        raise TypeError(f"{what}: expected a {dtype} tensor, got {sig[0]}")
    if sig[1] != shape:
        raise ValueError(f"{what} has shape {tuple(sig[1])}, expected {shape}")
    if sig[2][2] != 1 and sig[1][2] != 1:
        raise ValueError(f"{what}: a head's dims must be contiguous")
    return tuple(sig[2][i] if sig[1][i] > 1 else 0 for i in (0, 1))


@functools.lru_cache(maxsize=256)
def _rope_pos_plan(sig, inverse):
    """(descriptor by reference, storage type) of a call's tensors."""
    q, positions, k, q_out, k_out = sig
    if len(q[1]) != 3:
        raise ValueError("q has shape [heads, tokens, head_dim]")
    H, T, d = q[1]
    dt = _storage(q[0])
    _want(positions, torch.int32, (T,), "positions")
    Hk = 0
    if k is not None:
        if len(k[1]) != 3:
            raise ValueError("k has shape [heads, tokens, head_dim]")
        Hk = k[1][0]
    strides = (*_heads(q, q[0], (H, T, d), "q"), *_heads(q_out, q[0], (H, T, d), "q_out"),
               *_heads(k, q[0], (Hk, T, d), "k"), *_heads(k_out, q[0], (Hk, T, d), "k_out"))
    return C.byref(_abi.RopePosDesc(T, H, Hk, d, inverse, *strides)), dt


def rope_positions(q, positions, plan, k=None, inverse=False, q_out=None, k_out=None):
    """Rotary of q [H, T, d] (and k [Hk, T, d]) at positions (int32 [T] on the
    device) by a ``rope_plan``. Any strides with contiguous dims; a tensor
    [T, H, d] goes in transposed. q_out / k_out: where to (q and k themselves
    for in place; new tensors when None). Returns the result, or the two.
    inverse=True turns back (the gradient's call)."""
    if k is None and k_out is not None:
        raise ValueError("k_out given without k")
    ref = _plan_ref(plan)
    o = torch.empty_like(q) if q_out is None else q_out
    ko = torch.empty_like(k) if k_out is None and k is not None else k_out
    desc, dt = _rope_pos_plan(_sig(q, positions, k, o, ko), 1 if inverse else 0)
    dev = torch._C._cuda_getDevice()
    qp, pp, kp, op, lp = _addresses(dev, q, positions, k, o, ko)
    status = _lib().blk_rope_positions(desc, ref, qp, kp, pp, op, lp, dt,
                                       torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _abi.check(status, "blk_rope_positions")
    return o if k is None else (o, ko)


def _paged(dtype, k_cache, v_cache, k_scale, v_scale, block_table, lens):
    """Fields of blk_paged_desc, from the tensors' _sig."""
    if len(k_cache[1]) != 4:
        raise ValueError("k_cache has shape [pages, kv_heads, page_tokens, head_dim]")
    if len(block_table[1]) != 2:
        raise ValueError("block_table has shape [batch, max_pages]")
    pages, Hk, n, d = k_cache[1]
    B, max_pages = block_table[1]
    kind = _abi.BLK_CACHE_E4M3 if k_cache[0] is torch.float8_e4m3fn else _abi.BLK_CACHE_16BIT
    if kind == _abi.BLK_CACHE_16BIT and k_cache[0] is not dtype:
        raise TypeError(f"caches are float8_e4m3fn or {dtype}, got {k_cache[0]}")
    if (k_scale is None) != (kind == _abi.BLK_CACHE_16BIT) or (k_scale is None) != (v_scale is None):
        raise ValueError("a float8_e4m3fn cache has k_scale and v_scale, a 16-bit cache has none")
    _want(k_scale, torch.float32, (pages, Hk), "k_scale")
    _want(v_scale, torch.float32, (pages, Hk), "v_scale")
    if v_cache[0] is not k_cache[0] or v_cache[1] != k_cache[1]:
        raise ValueError("v_cache must be as k_cache")
    for c, what in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _dense((c[0], c[1][1:], c[2][1:]), f"a page of {what}")
    page_stride = Hk * n * d
    if pages > 1:
        page_stride = k_cache[2][0]
        if v_cache[2][0] != page_stride:
            raise ValueError("k_cache and v_cache must have the same page stride")
    _want(block_table, torch.int32, (B, max_pages), "block_table")
    _want(lens, torch.int32, (B,), "lens")
    return pages, n, Hk, d, B, max_pages, page_stride, kind


@functools.lru_cache(maxsize=256)
def _append_plan(sig):
    """(descriptor by reference, storage type) of a call's tensors."""
    k, v, q, q_out, cu_seqlens, positions, k_cache, v_cache, k_scale, v_scale, table, lens = sig
    if len(k[1]) != 3:
        raise ValueError("k has shape [kv_heads, tokens, head_dim]")
    Hk, T, d = k[1]
    dt = _storage(k[0])
    fields = _paged(k[0], k_cache, v_cache, k_scale, v_scale, table, lens)
    if fields[2] != Hk or fields[3] != d:
        raise ValueError(f"k has {Hk} heads of {d} dims, the cache {fields[2]} of {fields[3]}")
    _want(cu_seqlens, torch.int32, (fields[4] + 1,), "cu_seqlens")
    _want(positions, torch.int32, (T,), "positions")
    H = 0
    if q is not None:
        if len(q[1]) != 3:
            raise ValueError("q has shape [heads, tokens, head_dim]")
        H = q[1][0]
    strides = (*_heads(k, k[0], (Hk, T, d), "k"), *_heads(v, k[0], (Hk, T, d), "v"),
               *_heads(q, k[0], (H, T, d), "q"), *_heads(q_out, k[0], (H, T, d), "q_out"))
    return C.byref(_abi.AppendDesc(fields, T, H, *strides)), dt


def kv_append_paged(k, v, k_cache, v_cache, block_table, lens, cu_seqlens=None, k_scale=None,
                    v_scale=None, rope=None, positions=None, q=None, q_out=None):
    """Append new tokens' k and v [Hk, T, d] (any strides with contiguous dims; a
    tensor [T, Hk, d] goes in transposed) to paged caches [pages, Hk,
    page_tokens, d], in place: of the storage dtype, or float8_e4m3fn with
    scales fp32 [pages, Hk]. Sequence b's new tokens are rows cu_seqlens[b] ..
    cu_seqlens[b+1] - 1 (int32 [B + 1] on the device; None: row b) at the
    positions up to lens[b] - 1 (lens int32 [B]: with the new tokens), in pages
    block_table[b] (int32 [B, max_pages]). rope (a ``rope_plan``) turns k and q
    [H, T, d] on the way, at the positions in the cache or at ``positions``
    (int32 [T]). Returns q turned (q_out, or a new tensor; rows outside every
    sequence are not written), None without q."""
    if q is None and q_out is not None:
        raise ValueError("q_out given without q")
    ref = None if rope is None else _plan_ref(rope)
    o = torch.empty_like(q) if q_out is None and q is not None else q_out
    ts = (k, v, q, o, cu_seqlens, positions, k_cache, v_cache, k_scale, v_scale, block_table, lens)
    desc, dt = _append_plan(_sig(*ts))
    dev = torch._C._cuda_getDevice()
    kp, vp, qp, op, cup, pp, kcp, vcp, ksp, vsp, tp, lp = _addresses(dev, *ts)
    status = _lib().blk_kv_append_paged(desc, ref, kp, vp, qp, cup, pp, tp, lp, kcp, vcp, ksp, vsp,
                                        op, dt, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _abi.check(status, "blk_kv_append_paged")
    return o


def decode_paged_desc(fields, n_heads, q_batch_stride, q_head_stride, alibi=False, scale=None):
    """fields: those of blk_paged_desc in their order."""
    return _abi.DecodePagedDesc(fields, n_heads, q_batch_stride, q_head_stride,
                                -1.0 if scale is None else scale, 1 if alibi else 0)


def attn_decode_paged_workspace_size(desc) -> int:
    need = C.c_size_t(0)
    _abi.check(_lib().blk_attn_decode_paged_workspace_size(C.byref(desc), C.byref(need)),
               "blk_attn_decode_paged_workspace_size")
    return need.value


@functools.lru_cache(maxsize=256)
def _decode_paged_plan(sig, alibi, scale):
    """(descriptor by reference, workspace bytes, storage type) of a call's
    tensors and _values."""
    q, out, slopes, k_cache, v_cache, k_scale, v_scale, table, lens = sig
    if len(q[1]) != 3:
        raise ValueError("q has shape [batch, heads, head_dim]")
    B, H, d = q[1]
    dt = _storage(q[0])
    fields = _paged(q[0], k_cache, v_cache, k_scale, v_scale, table, lens)
    if fields[3] != d or fields[4] != B:
        raise ValueError(f"q {tuple(q[1])} does not fit the cache's head_dim {fields[3]} or "
                         f"block_table's {fields[4]} sequences")
    _want(slopes, torch.float32, (H,), "slopes")
    _want(out, q[0], (B, H, d), "out")
    desc = decode_paged_desc(fields, H, *_heads(q, q[0], (B, H, d), "q"), alibi, scale)
    return C.byref(desc), attn_decode_paged_workspace_size(desc), dt


def attn_decode_paged(q, k_cache, v_cache, block_table, lens, k_scale=None, v_scale=None,
                      alibi=False, slopes=None, scale=None, out=None, workspace=None):
    """One decode step over a paged cache: q [B, H, d] (newest token of each
    sequence, at position lens[b] - 1; any strides with contiguous dims)
    against caches [pages, Hk, page_tokens, d], in the storage dtype or
    float8_e4m3fn with scales fp32 [pages, Hk]; sequence b's keys 0 .. lens[b] -
    1 lie in pages block_table[b] (int32 [B, max_pages], lens int32 [B], both
    on the device). Length 0: a zero row. Returns o [B, H, d]."""
    ts = (q, out, slopes, k_cache, v_cache, k_scale, v_scale, block_table, lens)
    desc, need, dt = _decode_paged_plan(_sig(*ts), *_values(alibi, scale))
    dev = torch._C._cuda_getDevice()
    qp, op, sp, kp, vp, ksp, vsp, tp, lp = _addresses(dev, *ts)
    o = out
    if o is None:
        o = torch.empty_like(q) if q.is_contiguous() else torch.empty(q.shape, dtype=q.dtype, device=q.device)
        op = o.data_ptr()
    fn = _lib().blk_attn_decode_paged
    if need == 0 and workspace is None:
        status = fn(desc, qp, kp, vp, ksp, vsp, tp, lp, sp, op, None, 0, dt,
                    torch._C._cuda_getCurrentRawStream(dev))
    else:
        status = _with_workspace(
            lambda wp, wn, st: fn(desc, qp, kp, vp, ksp, vsp, tp, lp, sp, op, wp, wn, dt, st),
            workspace, need, dev)
    if status:
        _abi.check(status, "blk_attn_decode_paged")
    return o


def linear(x, w, bias=None, res1=None, res2=None, out=None):
    """y = x W^T [+ bias] [+ res1] [+ res2]; x [..., k], w [n, k]."""
    _same(x, w, bias, res1, res2, out)
    k = x.shape[-1]
    n = w.shape[0]
    m = x.numel() // k
    out = torch.empty((*x.shape[:-1], n), dtype=x.dtype, device=x.device) if out is None else out
    _abi.check(_lib().blk_linear(_p(x), _p(w), _p(bias), _p(res1), _p(res2), _p(out), m, n, k,
                                 _dt(x), _stream()), "blk_linear")
    return out


def q8_0_quantize(w):
    """Q8_0 of a weight w [n, k] (k % 32 == 0) on the GPU: (codes int8
    [n, k], scales fp16 [k/32, n], block-major)."""
    n, k = w.shape
    q = torch.empty((n, k), dtype=torch.int8, device=w.device)
    d = torch.empty((k // 32, n), dtype=torch.float16, device=w.device)
    _abi.check(_lib().blk_q8_0_quantize(_p(w), n, k, _p(q), _p(d), _dt(w), _stream()),
               "blk_q8_0_quantize")
    return q, d


def linear_q8_0(x, q, d, bias=None, res1=None, res2=None, out=None):
    """y = x W^T [+ bias] [+ res1] [+ res2] with W in Q8_0 form (q, d)."""
    _same(x, bias, res1, res2, out)
    if q.dtype != torch.int8 or d.dtype != torch.float16:
        raise TypeError("Q8_0 codes are int8 and scales fp16")
    k = x.shape[-1]
    n = q.shape[0]
    m = x.numel() // k
    out = torch.empty((*x.shape[:-1], n), dtype=x.dtype, device=x.device) if out is None else out
    _abi.check(_lib().blk_linear_q8_0(_p(x), _p(q), _p(d), _p(bias), _p(res1), _p(res2), _p(out),
                                      m, n, k, _dt(x), _stream()), "blk_linear_q8_0")
    return out


def mlp(x, w_up, w_down, w_gate=None, b_up=None, b_down=None, res1=None, res2=None,
        act="swiglu", workspace=None, out=None):
    """SwiGLU or GELU(tanh) MLP with optional biases and residual adds."""
    _same(x, w_up, w_down, w_gate, b_up, b_down, res1, res2, out)
    D = x.shape[-1]
    T = x.numel() // D
    F = w_up.shape[0]
    desc = _abi.MlpDesc(T, D, F, _abi.BLK_ACT_SWIGLU if act == "swiglu" else _abi.BLK_ACT_GELU_TANH)
    need = C.c_size_t(0)
    _abi.check(_lib().blk_mlp_workspace_size(C.byref(desc), C.byref(need)), "blk_mlp_workspace_size")
    if workspace is None:
        workspace = torch.empty(need.value, dtype=torch.uint8, device=x.device)
    out = torch.empty_like(x) if out is None else out
    _abi.check(_lib().blk_mlp(C.byref(desc), _p(x), _p(w_gate), _p(w_up), _p(b_up), _p(w_down),
                              _p(b_down), _p(res1), _p(res2), _p(out), _p(workspace),
                              workspace.numel(), _dt(x), _stream()), "blk_mlp")
    return out


def block_desc(cfg, batch: int, seq: int) -> _abi.BlockDesc:
    """Descriptor from a config object with the block's fields (hidden,
    n_heads, n_kv_heads, head_dim, intermediate, norm, norm_place, residual,
    eps, qkv_layout, qk_norm, qk_norm_eps, rotary_span, rope_base, alibi, act)."""
    q = _qkv_desc(batch, seq, cfg.hidden, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim,
                  cfg.qkv_layout, cfg.qk_norm, cfg.qk_norm_eps, cfg.rotary_span, cfg.rope_base)
    return _abi.BlockDesc(
        q,
        _abi.BLK_NORM_LAYERNORM if cfg.norm == "layernorm" else _abi.BLK_NORM_RMS,
        _abi.BLK_NORM_PRE if cfg.norm_place == "pre" else _abi.BLK_NORM_POST,
        _abi.BLK_RESIDUAL_SEQUENTIAL if cfg.residual == "sequential" else _abi.BLK_RESIDUAL_PARALLEL,
        cfg.eps, 1 if cfg.alibi else 0, cfg.intermediate,
        _abi.BLK_ACT_SWIGLU if cfg.act == "swiglu" else _abi.BLK_ACT_GELU_TANH)


def forward_workspace_size(cfg, batch: int, seq: int) -> int:
    desc = block_desc(cfg, batch, seq)
    need = C.c_size_t(0)
    _abi.check(_lib().blk_forward_workspace_size(C.byref(desc), C.byref(need)),
               "blk_forward_workspace_size")
    return need.value


def forward(cfg, weights: dict, x, workspace=None, out=None):
    """The block's prefill forward: x [B, S, D] -> y [B, S, D].

    weights maps slot names (``attn_norm_w``, ``w_qkv``, ...) to CUDA tensors;
    absent slots are NULL. workspace: a uint8 CUDA tensor of at least
    ``forward_workspace_size`` bytes (allocated here when None).
    """
    B, S, _ = x.shape
    desc = block_desc(cfg, B, S)
    ws_need = forward_workspace_size(cfg, B, S)
    if workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=x.device)
    unknown = set(weights) - set(_abi.WEIGHT_SLOTS)
    if unknown:
        raise KeyError(f"unknown weight slots: {sorted(unknown)}")
    for name, t in weights.items():
        if name != "alibi_slopes":
            _same(x, t)
    w = _abi.BlockWeights(*[_p(weights.get(n)) for n in _abi.WEIGHT_SLOTS])
    out = torch.empty_like(x) if out is None else out
    _abi.check(_lib().blk_forward(C.byref(desc), C.byref(w), _p(x), _p(out), _p(workspace),
                                  workspace.numel(), _dt(x), _stream()), "blk_forward")
    return out


def forward_packed_workspace_size(cfg, tokens: int, prompts: int) -> int:
    desc = block_desc(cfg, 1, tokens)
    need = C.c_size_t(0)
    _abi.check(_lib().blk_forward_packed_workspace_size(C.byref(desc), prompts, C.byref(need)),
               "blk_forward_packed_workspace_size")
    return need.value


def forward_packed(cfg, weights: dict, x, cu_seqlens, workspace=None, out=None):
    """The block over packed prompts: x [T, D] holds them one behind the other,
    prompt i in rows cu_seqlens[i] .. cu_seqlens[i+1] - 1 (int32 [prompts + 1]
    on the device). Returns y [T, D]; rows outside every prompt hold
    unspecified values. weights as for ``forward``."""
    T, D = x.shape
    if D != cfg.hidden:
        raise ValueError(f"x has {D} columns, the block {cfg.hidden}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens has shape [prompts + 1]")
    prompts = cu_seqlens.numel() - 1
    unknown = set(weights) - set(_abi.WEIGHT_SLOTS)
    if unknown:
        raise KeyError(f"unknown weight slots: {sorted(unknown)}")
    _same(x, out, *(t for name, t in weights.items() if name != "alibi_slopes"))
    _shape(out, (T, D), "out")
    desc = block_desc(cfg, 1, T)
    if workspace is None:
        workspace = torch.empty(forward_packed_workspace_size(cfg, T, prompts), dtype=torch.uint8,
                                device=x.device)
    w = _abi.BlockWeights(*[_p(weights.get(n)) for n in _abi.WEIGHT_SLOTS])
    out = torch.empty_like(x) if out is None else out
    dev = torch.cuda.current_device()
    (cup,) = _pointers(torch.int32, dev, cu_seqlens)
    wp, wn = _workspace(workspace, dev)
    xp, op = _pointers(x.dtype, dev, x, out)
    _abi.check(_lib().blk_forward_packed(C.byref(desc), C.byref(w), cup, prompts, xp, op, wp, wn,
                                         _dt(x), _stream()), "blk_forward_packed")
    return out


Q8_PROJECTIONS = ("qkv", "o", "gate", "up", "down")


def forward_q8_0_workspace_size(cfg, batch: int, seq: int) -> int:
    """Workspace bytes of blk_forward_q8_0's dequantize-once path."""
    desc = block_desc(cfg, batch, seq)
    need = C.c_size_t(0)
    _abi.check(_lib().blk_forward_q8_0_workspace_size(C.byref(desc), C.byref(need)),
               "blk_forward_q8_0_workspace_size")
    return need.value


def forward_q8_0(cfg, weights: dict, q8: dict, x, workspace=None, out=None):
    """The block with Q8_0 projection weights (blk_forward_q8_0). weights:
    the non-projection slots as for ``forward``; q8 maps ``q_<name>`` (int8
    codes) and ``d_<name>`` (fp16 scales) for name in qkv, o, gate, up, down
    (gate for SwiGLU only). workspace: ``forward_q8_0_workspace_size`` bytes
    (allocated here when None) take the dequantize-once path from 512 tokens
    on; ``forward_workspace_size`` bytes keep the W8A16 GEMMs."""
    B, S, _ = x.shape
    desc = block_desc(cfg, B, S)
    if workspace is None:
        workspace = torch.empty(forward_q8_0_workspace_size(cfg, B, S), dtype=torch.uint8,
                                device=x.device)
    unknown = set(weights) - set(_abi.WEIGHT_SLOTS)
    if unknown:
        raise KeyError(f"unknown weight slots: {sorted(unknown)}")
    unknown = set(q8) - set(_abi.Q8_SLOTS)
    if unknown:
        raise KeyError(f"unknown Q8_0 slots: {sorted(unknown)}")
    for name, t in weights.items():
        if name != "alibi_slopes":
            _same(x, t)
    for name, t in q8.items():
        want = torch.int8 if name.startswith("q_") else torch.float16
        if t.dtype != want or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name}: expected a contiguous CUDA {want} tensor")
    w = _abi.BlockWeights(*[_p(weights.get(n)) for n in _abi.WEIGHT_SLOTS])
    qw = _abi.Q8Weights(*[_p(q8.get(n)) for n in _abi.Q8_SLOTS])
    out = torch.empty_like(x) if out is None else out
    _abi.check(_lib().blk_forward_q8_0(C.byref(desc), C.byref(w), C.byref(qw), _p(x), _p(out),
                                       _p(workspace), workspace.numel(), _dt(x), _stream()),
               "blk_forward_q8_0")
    return out


def model_desc(cfg, batch: int, seq: int, n_layers: int, vocab: int, embed_norm: bool = False,
               final_norm: str = "layernorm", final_eps: float = 1e-5) -> _abi.ModelDesc:
    """Descriptor of an n_layers stack of cfg's block between the token
    embedding and the logits (blk_model_forward)."""
    return _abi.ModelDesc(block_desc(cfg, batch, seq), n_layers, vocab, 1 if embed_norm else 0,
                          _abi.BLK_NORM_LAYERNORM if final_norm == "layernorm" else _abi.BLK_NORM_RMS,
                          final_eps)


def model_workspace_size(cfg, batch: int, seq: int, n_layers: int, vocab: int, **kw) -> int:
    need = C.c_size_t(0)
    desc = model_desc(cfg, batch, seq, n_layers, vocab, **kw)
    _abi.check(_lib().blk_model_workspace_size(C.byref(desc), C.byref(need)),
               "blk_model_workspace_size")
    return need.value


_MODEL_SLOTS = ("embed", "embed_norm_w", "embed_norm_b", "layers", "final_norm_w",
                "final_norm_b", "lm_head")


def model_forward(cfg, model_w: dict, tokens, vocab: int, embed_norm: bool = False,
                  final_norm: str = "layernorm", final_eps: float = 1e-5, workspace=None,
                  out=None):
    """Token ids [B, S] (int32, CUDA) -> logits [B, S, vocab] in the storage
    dtype, through len(model_w["layers"]) blocks. model_w holds ``embed``
    [vocab, hidden], optional ``embed_norm_w``/``embed_norm_b``, ``layers``
    (a list of block weight dicts), ``final_norm_w``, optional
    ``final_norm_b`` and ``lm_head`` [vocab, hidden]."""
    unknown = set(model_w) - set(_MODEL_SLOTS)
    if unknown:
        raise KeyError(f"unknown model slots: {sorted(unknown)}")
    if tokens.dtype != torch.int32 or not tokens.is_cuda or tokens.dim() != 2:
        raise ValueError("tokens must be a CUDA int32 tensor [batch, seq]")
    B, S = tokens.shape
    emb = model_w["embed"]
    layers = model_w.get("layers", [])
    desc = model_desc(cfg, B, S, len(layers), vocab, embed_norm, final_norm, final_eps)
    need = model_workspace_size(cfg, B, S, len(layers), vocab, embed_norm=embed_norm,
                                final_norm=final_norm, final_eps=final_eps)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=tokens.device)
    arr = (_abi.BlockWeights * max(1, len(layers)))()
    for i, lw in enumerate(layers):
        bad = set(lw) - set(_abi.WEIGHT_SLOTS)
        if bad:
            raise KeyError(f"unknown weight slots in layer {i}: {sorted(bad)}")
        for name, t in lw.items():
            if name != "alibi_slopes":
                _same(emb, t)
        arr[i] = _abi.BlockWeights(*[_p(lw.get(n)) for n in _abi.WEIGHT_SLOTS])
    for n in ("embed_norm_w", "embed_norm_b", "final_norm_w", "final_norm_b", "lm_head"):
        _same(emb, model_w.get(n))
    mw = _abi.ModelWeights(_p(emb), _p(model_w.get("embed_norm_w")), _p(model_w.get("embed_norm_b")),
                           arr, _p(model_w.get("final_norm_w")), _p(model_w.get("final_norm_b")),
                           _p(model_w.get("lm_head")))
    out = torch.empty((B, S, vocab), dtype=emb.dtype, device=tokens.device) if out is None else out
    _same(emb, out)
    _abi.check(_lib().blk_model_forward(C.byref(desc), C.byref(mw), C.c_void_p(tokens.data_ptr()),
                                        _p(out), _p(workspace), workspace.numel(), _dt(emb),
                                        _stream()), "blk_model_forward")
    return out


def forward_host(cfg, weights: dict, x_host, y_host=None, x_dev=None, y_dev=None,
                 workspace=None, n_chunks=2):
    """The block on host tensors (pinned CPU memory), copies overlapped with
    compute over n_chunks groups of sequences. x_dev / y_dev / workspace are
    reusable device staging buffers (allocated here when None). Returns
    y_host; it is ready when the current stream reaches the end of the call."""
    if x_host.is_cuda or not x_host.is_pinned():
        raise ValueError("x_host must be a pinned CPU tensor")
    B, S, _ = x_host.shape
    dev = torch.device("cuda", torch.cuda.current_device())
    y_host = torch.empty_like(x_host).pin_memory() if y_host is None else y_host
    if y_host.is_cuda or not y_host.is_pinned() or y_host.shape != x_host.shape:
        raise ValueError("y_host must be a pinned CPU tensor shaped like x_host")
    x_dev = torch.empty(x_host.shape, dtype=x_host.dtype, device=dev) if x_dev is None else x_dev
    y_dev = torch.empty_like(x_dev) if y_dev is None else y_dev
    _same(x_host, x_dev, y_dev)
    desc = block_desc(cfg, B, S)
    ws_need = forward_workspace_size(cfg, B, S)
    if workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=dev)
    unknown = set(weights) - set(_abi.WEIGHT_SLOTS)
    if unknown:
        raise KeyError(f"unknown weight slots: {sorted(unknown)}")
    for name, t in weights.items():
        if name != "alibi_slopes":
            _same(x_host, t)
    w = _abi.BlockWeights(*[_p(weights.get(n)) for n in _abi.WEIGHT_SLOTS])
    _abi.check(_lib().blk_forward_host(C.byref(desc), C.byref(w), C.c_void_p(x_host.data_ptr()),
                                       C.c_void_p(y_host.data_ptr()), _p(x_dev), _p(y_dev),
                                       _p(workspace), workspace.numel(), n_chunks, _dt(x_host),
                                       _stream()), "blk_forward_host")
    return y_host


class HostPipe:
    """Block forwards over a stream of pinned host batches (blk_host_pipe_*):
    submit() enqueues one batch on the current stream and returns; batch n's
    copy in overlaps batch n-1's forward and its copy out batch n+1's.
    x_host must hold the batch at submit time; y_host is complete once the
    stream has passed a later flush(). Host tensors must stay alive until
    then; the pipe's device memory (staging slots and workspace) is
    allocated here."""

    def __init__(self, cfg, batch, seq, dtype=torch.bfloat16, depth=2):
        self.desc = block_desc(cfg, batch, seq)
        self.shape = (batch, seq, cfg.hidden)
        self.dtype = dtype
        n = C.c_size_t(0)
        _abi.check(_lib().blk_host_pipe_mem_size(C.byref(self.desc), depth, C.byref(n)),
                   "blk_host_pipe_mem_size")
        dev = torch.device("cuda", torch.cuda.current_device())
        self.mem = torch.empty(n.value, dtype=torch.uint8, device=dev)
        handle = C.c_void_p()
        dt = _abi.BLK_F16 if dtype == torch.float16 else _abi.BLK_BF16
        _abi.check(_lib().blk_host_pipe_create(C.byref(self.desc), depth, dt, _p(self.mem),
                                               n.value, C.byref(handle)), "blk_host_pipe_create")
        self._h = handle

    def submit(self, weights: dict, x_host, y_host):
        for t in (x_host, y_host):
            if t.is_cuda or not t.is_pinned() or tuple(t.shape) != self.shape or t.dtype != self.dtype:
                raise ValueError(f"host batches must be pinned CPU tensors {self.shape} {self.dtype}")
        unknown = set(weights) - set(_abi.WEIGHT_SLOTS)
        if unknown:
            raise KeyError(f"unknown weight slots: {sorted(unknown)}")
        w = _abi.BlockWeights(*[_p(weights.get(n)) for n in _abi.WEIGHT_SLOTS])
        _abi.check(_lib().blk_host_pipe_submit(self._h, C.byref(w), C.c_void_p(x_host.data_ptr()),
                                               C.c_void_p(y_host.data_ptr()), _stream()),
                   "blk_host_pipe_submit")

    def flush(self):
        _abi.check(_lib().blk_host_pipe_flush(self._h, _stream()), "blk_host_pipe_flush")

    def close(self):
        if self._h:
            _abi.check(_lib().blk_host_pipe_destroy(self._h), "blk_host_pipe_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class ForwardGraph:
    """The block forward recorded once as a CUDA graph (blk_forward_graph_create)
    for fixed tensors x, y, workspace and weights; launch() replays it on the
    current stream. The tensors must stay alive while the graph is used."""

    def __init__(self, cfg, weights: dict, x, y, workspace, events=None):
        B, S, _ = x.shape
        self._keep = (weights, x, y, workspace)
        self.desc = block_desc(cfg, B, S)
        unknown = set(weights) - set(_abi.WEIGHT_SLOTS)
        if unknown:
            raise KeyError(f"unknown weight slots: {sorted(unknown)}")
        for name, t in weights.items():
            if name != "alibi_slopes":
                _same(x, t)
        _same(x, y)
        self.w = _abi.BlockWeights(*[_p(weights.get(n)) for n in _abi.WEIGHT_SLOTS])
        ev = None
        n_ev = 0
        if events:
            ev = (C.c_void_p * len(events))(*[e.cuda_event for e in events])
            n_ev = len(events)
        self.kinds = (C.c_int32 * 12)()  # a block makes at most 12 launches
        self.n_launches = C.c_int(0)
        handle = C.c_void_p()
        _abi.check(_lib().blk_forward_graph_create(C.byref(self.desc), C.byref(self.w), _p(x), _p(y),
                                                   _p(workspace), workspace.numel(), _dt(x), ev,
                                                   n_ev, self.kinds, C.byref(self.n_launches),
                                                   C.byref(handle)), "blk_forward_graph_create")
        self._h = handle

    def launch(self, events=None):
        """Replay on the current stream; events (torch.cuda.Event, created) replace
        the recorded ones for this and later launches."""
        if events is not None:
            arr = (C.c_void_p * len(events))(*[e.cuda_event for e in events])
            _abi.check(_lib().blk_graph_set_events(self._h, arr, len(events)),
                       "blk_graph_set_events")
        _abi.check(_lib().blk_graph_launch(self._h, _stream()), "blk_graph_launch")

    def close(self):
        if self._h:
            _abi.check(_lib().blk_graph_destroy(self._h), "blk_graph_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def check_device_status():
    """Synchronise the current stream and raise if an in-kernel wait timed out."""
    _abi.check(_lib().blk_check_device_status(_stream()), "blk_check_device_status")
