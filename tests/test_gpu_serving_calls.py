"""The packed and shared-prefix calls as a serving loop makes them (GPU): the
packed block captured and replayed, calls on two streams at once."""
import dataclasses

import pytest
import torch

import alibi_attention_block_gb300 as blk
import workloads
from tests.parity import to_dev
from tests.test_gpu_packed import BLOCKS, ends, inputs as packed_inputs, table
from tests.test_gpu_shared import inputs as shared_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


@pytest.mark.parametrize("name", sorted(BLOCKS))
@pytest.mark.parametrize("empty", [0, 300])
def test_captured_block(name, empty):
    """A captured block follows new tables and inputs, with its work list in
    shared memory or (empty prompts) in the graph's workspace; other calls
    between its replays do not touch it."""
    T = 400
    cfg = dataclasses.replace(BLOCKS[name], seq=T)
    x, w = workloads.block_inputs(cfg)
    x, wd = to_dev(x)[0], {n: to_dev(t) for n, t in w.items()}
    cu = table([0, 70, 271, T] + [T] * empty)
    blk.forward_packed(cfg, wd, x, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = blk.forward_packed(cfg, wd, x, cu)
    for tab in ([0, 70, 271, T], [0, 1, 130, T], [0, T, T, T]):
        cu.copy_(table(tab + [T] * empty))
        x.copy_(x.flip(0))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        blk.forward_packed(cfg, wd, x.flip(0).contiguous(), cu)
        want = blk.forward_packed(cfg, wd, x, cu)
        blk.check_device_status()
        assert torch.equal(got, want)
        assert torch.equal(y, got)


def test_two_streams_at_once():
    """Calls without workspaces of their own, alternating on two streams."""
    lens = [100, 257, 1, 300]
    cu = [table(ends(lens) + [sum(lens)] * n) for n in (0, 300)]
    pre = [to_dev(t) for t in packed_inputs(8, 2, sum(lens), 128, 130, "bf16", 71)]
    step = [to_dev(t) for t in shared_inputs(6, 8, 2, 128, 3000, 200, "bf16", 72)]
    few = [to_dev(t) for t in shared_inputs(4, 8, 2, 64, 100, 60, "bf16", 73)]
    n6 = torch.tensor([200, 1, 90, 0, 30, 128], dtype=torch.int32, device="cuda")
    n4 = torch.tensor([60, 1, 0, 17], dtype=torch.int32, device="cuda")
    calls = [lambda i=i: blk.attn_prefill_packed(*pre[:3], cu[i], k_prefix=pre[3], v_prefix=pre[4]) for i in (0, 1)]
    calls += [lambda: blk.attn_decode_shared(*step, n6), lambda: blk.attn_decode_shared(*few, n4)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for r in range(12):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                i = (r + j) % len(calls)
                got.append((i, calls[i]()))
    torch.cuda.synchronize()
    blk.check_device_status()
    for i, o in got:
        assert torch.equal(o, want[i]), f"call {i}"
