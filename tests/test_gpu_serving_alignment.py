"""The packed and shared-prefix calls with tensors and workspaces that have the
16-byte alignment that the library asks for, and no more (GPU)."""
import dataclasses

import pytest
import torch

import alibi_attention_block_gb300 as blk
import workloads
from tests.parity import to_dev
from tests.test_gpu_packed import BLOCKS, ends, inputs as packed_inputs, table
from tests.test_gpu_shared import inputs as shared_inputs

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def at_16(t):
    """A copy of t whose address is 16 behind a boundary of 32."""
    if t is None:
        return None
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
    out = flat[8:8 + t.numel()].view(t.shape)
    assert out.data_ptr() % 32 == 16 and out.is_contiguous()
    return out.copy_(t)


class Workspace:
    """A workspace of n bytes at such an address, between guards."""

    def __init__(self, n):
        self.all = torch.full((n + 2 * GUARD + 32,), 0xA5, dtype=torch.uint8, device="cuda")
        first = GUARD + 16
        self.ws = self.all[first:first + n]
        assert n == 0 or self.ws.data_ptr() % 32 == 16
        self.first, self.end = first, first + n

    def check(self):
        assert (self.all[:self.first] == 0xA5).all() and (self.all[self.end:] == 0xA5).all()


@pytest.mark.parametrize("B,H,Hk,d,P,S", [
    (3, 4, 4, 64, 100, 40), (2, 8, 2, 128, 50, 70),                    # few keys
    (5, 8, 8, 64, 3000, 300), (40, 16, 2, 64, 700, 200), (5, 8, 8, 128, 1000, 300), (70, 8, 2, 128, 400, 129),
    (6, 8, 4, 128, 0, 900)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_shared(B, H, Hk, d, P, S, dt):
    q, kp, vp, k, v = shared_inputs(B, H, Hk, d, P, S, dt, 61)
    args = [to_dev(t) for t in (q, kp, vp, k, v)]
    lens = torch.tensor([1 + (31 * i) % S for i in range(B)], dtype=torch.int32, device="cuda")
    want = blk.attn_decode_shared(*args, lens)
    blk.check_device_status()
    w = Workspace(blk.attn_decode_shared_workspace_size(blk.decode_shared_desc(B, S, H, Hk, d, P)))
    out = at_16(torch.zeros_like(want))
    blk.attn_decode_shared(*map(at_16, args), lens, out=out, workspace=w.ws)
    blk.check_device_status()
    assert torch.equal(out, want)
    w.check()


@pytest.mark.parametrize("H,Hk,d,P,alibi", [
    (2, 2, 64, 100, False), (4, 2, 64, 0, True), (2, 2, 128, 70, False), (8, 2, 128, 0, False),
    (8, 2, 128, 100, True), (2, 2, 160, 0, True), (8, 2, 160, 130, False)])
@pytest.mark.parametrize("empty", [0, 300])
def test_packed(H, Hk, d, P, alibi, empty):
    lens = [100, 257, 1, 300]
    cu = table(ends(lens) + [sum(lens)] * empty)
    q, k, v, kp, vp = map(to_dev, packed_inputs(H, Hk, sum(lens), d, P, "bf16", 62))
    want = blk.attn_prefill_packed(q, k, v, cu, k_prefix=kp, v_prefix=vp, alibi=alibi)
    blk.check_device_status()
    w = Workspace(blk.attn_prefill_packed_workspace_size(
        blk.packed_desc(sum(lens), len(lens) + empty, H, Hk, d, P, alibi)))
    out = at_16(torch.zeros_like(want))
    blk.attn_prefill_packed(*map(at_16, (q, k, v)), cu, k_prefix=at_16(kp), v_prefix=at_16(vp), alibi=alibi,
                            out=out, workspace=w.ws)
    blk.check_device_status()
    assert torch.equal(out, want)
    w.check()


@pytest.mark.parametrize("name", sorted(BLOCKS))
@pytest.mark.parametrize("empty", [0, 300])
def test_block(name, empty):
    lens = [70, 1, 0, 200]
    cfg = dataclasses.replace(BLOCKS[name], seq=sum(lens))
    x, w = workloads.block_inputs(cfg)
    x, wd = to_dev(x)[0], {n: to_dev(t) for n, t in w.items()}
    cu = table(ends(lens) + [sum(lens)] * empty)
    want = blk.forward_packed(cfg, wd, x, cu)
    blk.check_device_status()
    ws = Workspace(blk.forward_packed_workspace_size(cfg, sum(lens), len(lens) + empty))
    out = at_16(torch.zeros_like(want))
    blk.forward_packed(cfg, wd, at_16(x), cu, workspace=ws.ws, out=out)
    blk.check_device_status()
    assert torch.equal(out, want)
    ws.check()
