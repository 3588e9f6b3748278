"""The Python binding's cached call plans (descriptor and workspace size),
without a GPU: the launch is replaced by a recorder, everything before it runs."""
import pytest
import torch

import alibi_attention_block_gb300 as blk
from alibi_attention_block_gb300 import build


class Recorder:
    """The library with its two launches replaced: they note the descriptor."""

    def __init__(self, lib):
        self._lib, self.descs = lib, []

    def __getattr__(self, name):
        if name in ("blk_attn_prefill_packed", "blk_attn_decode_shared"):
            return self._record
        return getattr(self._lib, name)

    def _record(self, desc, *args):
        d = desc._obj
        self.descs.append((d.softmax_scale, d.alibi))
        return 0


@pytest.fixture()
def recorder(monkeypatch):
    build.build()
    rec = Recorder(blk._lib())
    monkeypatch.setattr(blk, "_lib", lambda: rec)
    monkeypatch.setattr(blk, "_pointers", lambda dtype, dev, *ts: [None if t is None else 1 << 20 for t in ts])
    monkeypatch.setattr(blk, "_with_workspace", lambda call, workspace, need, dev: call(None, 0, 0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return rec


def packed(**kw):
    q, k = torch.zeros(4, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    blk.attn_prefill_packed(q, k, k, torch.tensor([0, 8], dtype=torch.int32), **kw)


def shared(**kw):
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 8, 64, dtype=torch.bfloat16)
    blk.attn_decode_shared(q, None, None, k, k, torch.ones(3, dtype=torch.int32), **kw)


@pytest.mark.parametrize("call", [packed, shared])
def test_a_scale_changed_in_place_is_seen(recorder, call):
    """A 0-dim tensor as scale stands for its value at the call."""
    scale = torch.tensor(0.25)
    call(scale=scale)
    scale.mul_(2)
    call(scale=scale)
    call(scale=0.25)
    call()
    assert [s for s, _ in recorder.descs] == [0.25, 0.5, 0.25, -1.0]


@pytest.mark.parametrize("call", [packed, shared])
def test_an_alibi_switch_changed_in_place_is_seen(recorder, call):
    alibi = torch.tensor(True)
    call(alibi=alibi)
    alibi.fill_(False)
    call(alibi=alibi)
    assert [a for _, a in recorder.descs] == [1, 0]


@pytest.mark.parametrize("call,plan", [(packed, "_packed_plan"), (shared, "_decode_shared_plan")])
def test_plans_keep_no_tensor(recorder, call, plan):
    """Calls with tensors of one value share one plan."""
    getattr(blk, plan).cache_clear()
    for _ in range(3):
        call(scale=torch.tensor(0.125), alibi=torch.tensor(False))
    call(scale=0.125)
    assert getattr(blk, plan).cache_info().currsize == 1


@pytest.mark.parametrize("call", [packed, shared])
def test_a_scale_that_cannot_be_hashed(recorder, call):
    """An array of one element is taken for its value, as by the dense calls."""
    np = pytest.importorskip("numpy")
    call(scale=np.array(0.5))
    assert recorder.descs[-1][0] == 0.5
