"""The paged cache as a serving loop uses it: prompts projected, turned and appended, then decode
steps, each one append and one attention, against the oracle's attention over the history in 64 bits."""
import numpy as np
import pytest
import torch

import alibi_attention_block_gb300 as blk
import oracle
from tests import paged_ref as ref
from tests.parity import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bits,H,Hk,d,span,page", [(8, 8, 2, 128, 128, 16), (16, 4, 4, 64, 16, 32), (8, 4, 1, 160, 40, 64)])
@pytest.mark.parametrize("graph", [False, True])
def test_prompts_then_steps(bits, H, Hk, d, span, page, graph):
    """Three prompts, one of them in two chunks, then 40 steps. The caches' errors (half a step of
    the type for each key and value, e4m3: 2^-4) are let into the history that the oracle sees: the
    cache is read back; what remains is the attention's own error, as in test_gpu_paged.py. That the
    cache holds the projected, turned keys is checked apart, against the projection in 64 bits."""
    hidden, prompts = 256, [37, 90, 1]
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    w = (torch.randn(((H + 2 * Hk) * d, hidden), generator=g, device="cuda") * hidden ** -0.5).bfloat16()
    plan = blk.rope_plan(span, 10000.0)
    B, pages = 3, 64
    kind = torch.float8_e4m3fn if bits == 8 else torch.bfloat16
    kc, vc = (torch.zeros((pages, Hk, page, d), device="cuda").to(kind) for _ in "kv")
    ks, vs = (torch.zeros((pages, Hk), device="cuda") for _ in "kv") if bits == 8 else (None, None)
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    order = np.random.RandomState(3).permutation(pages)
    for b in range(B):
        table[b, :12] = i32(order[12 * b:12 * b + 12].tolist())
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    keys = [[] for _ in range(B)]  # projected keys in 64 bits, turned

    def project(x, positions, of):
        """q [H, T, d], k, v [Hk, T, d] of rows x [T, hidden]; notes the keys."""
        q, k, v = blk.qkv_bias_rope_partial(x[None], w, n_heads=H, n_kv_heads=Hk, head_dim=d)
        kt, _ = ref.turn(f64(k[0].float()), positions, ref.thetas(span), False)
        for t, b in enumerate(of):
            keys[b].append(kt[:, t])
        return q[0], k[0], v[0]

    def rows(n):
        return torch.randn((n, hidden), generator=g, device="cuda").bfloat16()

    # prompts: the first 60 tokens of prompt 1 in one call, the rest, and the others, in a second
    for chunk in ([0, 60, 0], [37, 30, 1]):
        start = lens.tolist()
        pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, chunk)])
        q, k, v = project(rows(sum(chunk)), pos, [b for b, n in enumerate(chunk) for _ in range(n)])
        lens += i32(chunk)
        qa = blk.kv_append_paged(k, v, kc, vc, table, lens, cu_seqlens=i32(np.concatenate([[0], np.cumsum(chunk)]).tolist()),
                                 k_scale=ks, v_scale=vs, rope=plan, q=q)
        # the queries turned on the way are those of the rotary by itself
        assert torch.equal(qa, blk.rope_positions(q, i32(pos.tolist()), plan))
    assert lens.tolist() == prompts

    x = rows(B)
    q, k, v = (torch.zeros((n, B, d), dtype=torch.bfloat16, device="cuda") for n in (H, Hk, Hk))
    o = torch.zeros((B, H, d), dtype=torch.bfloat16, device="cuda")

    def step():
        lens.add_(1)
        turned = blk.kv_append_paged(k, v, kc, vc, table, lens, k_scale=ks, v_scale=vs, rope=plan, q=q)
        blk.attn_decode_paged(turned.transpose(0, 1), kc, vc, table, lens, k_scale=ks, v_scale=vs, out=o)

    recorded = None
    for i in range(40):
        x = rows(B)
        qn, kn, vn = project(x, lens.tolist(), range(B))
        for a, b in ((q, qn), (k, kn), (v, vn)):
            a.copy_(b)
        if graph and recorded is None:
            recorded = torch.cuda.CUDAGraph()
            with torch.cuda.graph(recorded):
                step()
        recorded.replay() if graph else step()
        torch.cuda.synchronize()
        if i % 13 and i != 39:
            continue
        qt = f64(blk.rope_positions(q, lens - 1, plan).float())
        for b, n in enumerate(lens.tolist()):
            kr, seen, _ = ref.rows(kc, ks, table[b].tolist(), n, page)
            vr, _, _ = ref.rows(vc, vs, table[b].tolist(), n, page)
            assert seen.all() and n == prompts[b] + i + 1
            want, mag = (oracle.attention_decode(qt[None, :, b], kr[None], z[None], [n])[0] for z in (vr, np.abs(vr)))
            bound = (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * np.abs(want) + n * 2.0 ** -20 * np.abs(vr).max()
            assert (np.abs(f64(o[b].float()) - want) <= bound).all(), f"step {i} row {b}"
            # the cache: half a step of its type off (a growing scale's second rounding: below 2^-6 of the largest
            # code only), and the turn's 2^-20
            true = np.stack(keys[b], 1)
            half = 2.0 ** -4 if bits == 8 else 2.0 ** -8
            least = 2.0 ** -9 * float(ks.max()) if bits == 8 else 0.0
            assert (np.abs(kr - true) <= half * np.abs(true) + least + 2.0 ** -18 * np.abs(true).max()).all()
    blk.check_device_status()
