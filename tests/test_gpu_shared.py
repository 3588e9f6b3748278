"""GPU parity of blk_attn_decode_shared (one decode step of a batch whose
sequences share a prefix) against the fp64 oracle, through the C ABI.

Error bound of one output element, as in test_gpu_packed.py (u = eps / 2 of
the storage type, half a step): the prefix's weights are rounded once to the
storage type, the own cache's are not, the output is rounded once, and the
fp32 parts (scores, exponentials, sums, the merge) add less than 2^-14
relative:
    |err| <= (u + 2^-14) sum_j p_j |v_j| + u |o| + n 2^-25 max |v|.
"""
import numpy as np
import pytest
import torch

import alibi_attention_block_gb300 as blk
import oracle
from tests.parity import f64, to_dev
from tests.test_gpu_packed import HALF_STEP, slopes_of
from workloads import draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from alibi_attention_block_gb300 import build
    build.build()


def inputs(B, H, Hk, d, P, S, dt, seed):
    q, k, v = draw((B, H, d), dt, seed), draw((B, Hk, S, d), dt, seed + 1), draw((B, Hk, S, d), dt, seed + 2)
    kp = draw((Hk, P, d), dt, seed + 3) if P else None
    vp = draw((Hk, P, d), dt, seed + 4) if P else None
    return q, kp, vp, k, v


def check(got, q, kp, vp, k, v, lens, dt, slopes=None, scale=None, name=""):
    """Every row against the oracle's decode over prefix + own cache."""
    P = 0 if kp is None else kp.shape[1]
    u = HALF_STEP[dt]
    got = f64(got)
    for b, n in enumerate(lens):
        if n == 0:
            assert not got[b].any(), f"{name} row {b} is not zero"
            continue
        kb, vb = f64(k[b:b + 1, :, :n]), f64(v[b:b + 1, :, :n])
        if P:
            kb, vb = np.concatenate([f64(kp)[None], kb], 2), np.concatenate([f64(vp)[None], vb], 2)
        o, a = (oracle.attention_decode(f64(q[b:b + 1]), kb, w, [P + n], scale=scale, slopes=slopes)[0]
                for w in (vb, np.abs(vb)))
        bound = (u + 2.0 ** -14) * a + u * np.abs(o) + (P + n) * 2.0 ** -25 * np.abs(vb).max()
        err = np.abs(got[b] - o)
        assert np.isfinite(got[b]).all(), f"{name} row {b}: non-finite output"
        assert (err <= bound).all(), \
            f"{name} row {b}: error {err.max():.3e}, {float((err / bound).max()):.2f} of the bound"


CASES = [
    # B, H, Hk, d, prefix, max_seq, lens, alibi, dtype
    (1, 2, 2, 64, 1, 1, [1], False, "bf16"),
    (3, 4, 4, 64, 500, 64, [1, 64, 33], True, "fp16"),
    (2, 4, 2, 64, 128, 70, [70, 0], False, "fp16"),
    (5, 8, 2, 128, 129, 40, [1, 2, 0, 40, 39], False, "bf16"),
    (40, 8, 1, 128, 300, 9, [1 + i % 9 for i in range(40)], True, "bf16"),   # three row tiles, the last part-filled
    (130, 2, 2, 64, 257, 5, [i % 6 for i in range(130)], False, "bf16"),     # two row tiles of 128 sequences
    (33, 8, 2, 64, 1000, 3, [3] * 33, True, "bf16"),
    (2, 16, 16, 128, 4100, 130, [130, 5], False, "fp16"),
    (2, 4, 4, 128, 127, 300, [300, 17], True, "fp16"),
    (4, 8, 1, 64, 2500, 200, [200, 1, 77, 128], True, "fp16"),
    (3, 4, 1, 128, 0, 100, [100, 0, 1], True, "bf16"),                       # no prefix
    (2, 32, 8, 128, 20000, 64, [64, 1], False, "bf16"),
    (1, 6, 6, 64, 700, 10, [4], True, "bf16"),                               # given slopes
    (1500, 2, 2, 64, 40, 3, [i % 4 for i in range(1500)], False, "bf16"),    # many sequences, some away
    (1100, 8, 1, 128, 0, 2, [i % 3 for i in range(1100)], True, "fp16"),
]


ROOM = 800  # more capacity than the kernel for few keys takes, at any head_dim


def test_room_chooses_the_kernel():
    """Few keys need no workspace; the same with ROOM more capacity do."""
    for d in (64, 128):
        assert blk.attn_decode_shared_workspace_size(blk.decode_shared_desc(2, 20, 4, 2, d, 100)) == 0
        assert blk.attn_decode_shared_workspace_size(blk.decode_shared_desc(2, 20 + ROOM, 4, 2, d, 0)) > 0


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}H{}Hk{}d{}P{}S{}{}_{}".format(
    *c[:6], "_alibi" if c[7] else "", c[8]))
def test_shared_matches_oracle(case, room):
    """With capacity to spare, every case goes to the kernel for many keys."""
    B, H, Hk, d, P, S, lens, alibi, dt = case
    q, kp, vp, k, v = inputs(B, H, Hk, d, P, S, dt, 300 + B + H + d + P)
    kd, vd = (torch.zeros((B, Hk, S + room, d), dtype=t.dtype, device="cuda") for t in (k, v))
    kd[:, :, :S], vd[:, :, :S] = to_dev(k), to_dev(v)
    for b, n in enumerate(lens):  # entries past each length are not part of the sequence
        kd[b, :, n:] = float("nan")
        vd[b, :, n:] = float("nan")
    ref_slopes, dev_slopes = slopes_of(H, alibi)
    o = blk.attn_decode_shared(to_dev(q), to_dev(kp), to_dev(vp), kd, vd,
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), alibi=alibi,
                               slopes=dev_slopes)
    blk.check_device_status()
    check(o, q, kp, vp, k, v, lens, dt, ref_slopes, name=str(case))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_every_kernel(dt, d, G):
    """Each instantiation: several segments of prefix and own caches per CTA
    and per unit, tails of every kind, with and without ALiBi."""
    B, Hk, P, S = 21, 4, 1500, 300
    q, kp, vp, k, v = inputs(B, Hk * G, Hk, d, P, S, dt, 400 + d + G)
    lens = [(97 * i) % (S + 1) for i in range(B)]
    args = [to_dev(t) for t in (q, kp, vp, k, v)] + [torch.tensor(lens, dtype=torch.int32, device="cuda")]
    for alibi in (False, True):
        ref_slopes, dev_slopes = slopes_of(Hk * G, alibi)
        o = blk.attn_decode_shared(*args, alibi=alibi, slopes=dev_slopes)
        blk.check_device_status()
        check(o, q, kp, vp, k, v, lens, dt, ref_slopes, name=f"alibi {alibi}")


def test_own_caches_beyond_32_bit_offsets():
    """Caches of more than 2^31 elements: the last sequences' own keys lie
    behind the range of 32-bit offsets."""
    B, H, Hk, d, P, S = 9, 4, 2, 128, 150, (1 << 31) // (8 * 2 * 128) + 1000
    q, kp, vp, k, v = inputs(B, H, Hk, d, P, 300, "bf16", 77)
    kd, vd = (torch.zeros((B, Hk, S, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kd[:, :, :300], vd[:, :, :300] = to_dev(k), to_dev(v)
    assert kd.numel() > 1 << 31 and (B - 1) * Hk * S * d > 1 << 31
    lens = [300, 1, 2, 128, 129, 17, 255, 0, 300]
    o = blk.attn_decode_shared(to_dev(q), to_dev(kp), to_dev(vp), kd, vd,
                               torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check(o, q, kp, vp, k, v, lens, "bf16", name="long caches")


@pytest.mark.parametrize("d,P", [(64, 1200), (128, 1200), (64, 600), (128, 300)])
def test_growing_scores_rescale(d, P):
    """Scores that rise or fall along the prefix move the running maximum at
    every tile in one direction or the other."""
    B, H, S = 3, 2, 40
    q, kp, vp, k, v = inputs(B, H, H, d, P, S, "bf16", 8)
    q = torch.ones_like(q)
    for ramp in (torch.linspace(0, 3, P), torch.linspace(3, 0, P)):
        kp = (ramp[:, None] * torch.ones(H, P, d)).to(torch.bfloat16)
        o = blk.attn_decode_shared(*(to_dev(t) for t in (q, kp, vp, k, v)),
                                   torch.tensor([40, 1, 7], dtype=torch.int32, device="cuda"))
        check(o, q, kp, vp, k, v, [40, 1, 7], "bf16", name=f"d {d}")


def test_equals_decode_over_copied_prefix():
    """blk_attn_decode with the prefix copied in front of every cache says
    nearly the same (its weights are not rounded), as does a long prefix cut
    anywhere between shared and own."""
    B, H, Hk, d, P, S = 3, 8, 2, 64, 900, 100
    q, kp, vp, k, v = inputs(B, H, Hk, d, P, S, "bf16", 21)
    lens = [100, 1, 50]
    qd, kpd, vpd, kd, vd = map(to_dev, (q, kp, vp, k, v))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    full_k, full_v = (torch.cat([p.expand(B, -1, -1, -1), c], 2).contiguous() for p, c in ((kpd, kd), (vpd, vd)))
    one = blk.attn_decode(qd, full_k, full_v, n + P, alibi=True)
    check(one, q, kp, vp, k, v, lens, "bf16", oracle.alibi_slopes(H), name="copied prefix")
    for cut in (900, 640, 1):
        o = blk.attn_decode_shared(qd, kpd[:, :cut].contiguous(), vpd[:, :cut].contiguous(),
                                   full_k[:, :, cut:].contiguous(), full_v[:, :, cut:].contiguous(),
                                   n + (P - cut), alibi=True)
        check(o, q, kp, vp, k, v, lens, "bf16", oracle.alibi_slopes(H), name=f"cut at {cut}")


@pytest.mark.parametrize("P", [700, 1400])
def test_lengths_clamped_and_deterministic(P):
    B, H, d, S = 3, 4, 64, 32
    t = [to_dev(x) for x in inputs(B, H, H, d, P, S, "bf16", 31)]

    def call(lens):
        return blk.attn_decode_shared(*t, torch.tensor(lens, dtype=torch.int32, device="cuda"))

    a, b = call([-5, 32, 99]), call([0, 32, 32])
    assert torch.equal(a, b) and not a[0].any()
    assert torch.equal(call([7, 8, 9]), call([7, 8, 9]))


@pytest.mark.parametrize("B,H,Hk,d,P,S", [
    (64, 16, 4, 128, 16384, 256), (64, 8, 8, 64, 16384, 256), (64, 8, 8, 128, 16384, 256),
    (256, 4, 4, 64, 5000, 20), (200, 4, 1, 64, 20000, 20),
    # three row tiles per kv head and many kv heads: CTAs pass through several
    # units, with and without a second row tile
    (300, 200, 200, 64, 100, 3), (257, 160, 160, 128, 200, 3), (72, 320, 40, 128, 400, 3)])
def test_back_to_back(B, H, Hk, d, P, S):
    """Every query row in use and many key tiles per CTA, so that the two
    streams run far apart while loads are late: 25 steps without a pause give
    the same bits, and rows of them are the oracle's."""
    q, kp, vp, k, v = inputs(B, H, Hk, d, P, S, "bf16", 91)
    lens = [1 + (37 * i) % S for i in range(B)]
    args = [to_dev(t) for t in (q, kp, vp, k, v)] + [torch.tensor(lens, dtype=torch.int32, device="cuda")]
    outs = [blk.attn_decode_shared(*args) for _ in range(25)]
    blk.check_device_status()
    assert all(torch.equal(o, outs[0]) for o in outs)
    for b in (0, B // 2 - 3, B - 1):
        check(outs[0][b:b + 1], q[b:b + 1], kp, vp, k[b:b + 1], v[b:b + 1], lens[b:b + 1], "bf16", name=f"row {b}")


def test_scale_and_workspace():
    B, H, Hk, d, P, S = 4, 8, 8, 128, 400, 20
    q, kp, vp, k, v = inputs(B, H, Hk, d, P, S, "fp16", 41)
    lens = [20, 1, 2, 3]
    ws = torch.full((blk.attn_decode_shared_workspace_size(blk.decode_shared_desc(B, S, H, Hk, d, P)),),
                    255, dtype=torch.uint8, device="cuda")  # NaN wherever nothing is written
    out = torch.empty((B, H, d), dtype=torch.float16, device="cuda")
    o = blk.attn_decode_shared(*(to_dev(t) for t in (q, kp, vp, k, v)),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=0.2,
                               out=out, workspace=ws)
    assert o is out
    check(o, q, kp, vp, k, v, lens, "fp16", scale=np.float32(0.2), name="scale")


@pytest.mark.parametrize("P", [100, 1000])
def test_graph_replay_and_other_stream(P):
    B, H, Hk, d, S = 6, 8, 2, 128, 50
    qd, kpd, vpd, kd, vd = (to_dev(t) for t in inputs(B, H, Hk, d, P, S, "bf16", 51))
    lens = torch.tensor([50, 1, 2, 0, 30, 7], dtype=torch.int32, device="cuda")
    ws = torch.empty(blk.attn_decode_shared_workspace_size(blk.decode_shared_desc(B, S, H, Hk, d, P)),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(qd)

    def call():
        return blk.attn_decode_shared(qd, kpd, vpd, kd, vd, lens, out=out, workspace=ws)

    first = call().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
        assert torch.equal(out, first)
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.synchronize()
    for new in ([1, 50, 50, 3, 0, 9], [0, 0, 0, 0, 0, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        qd.copy_(qd.flip(0))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, blk.attn_decode_shared(qd, kpd, vpd, kd, vd, lens))


def test_captured_without_a_workspace():
    """A captured call takes its workspace from the graph's memory: other calls
    between its replays, and a second graph's, do not touch it."""
    B, H, Hk, d, P, S = 6, 8, 2, 128, 1000, 50
    args = [to_dev(t) for t in inputs(B, H, Hk, d, P, S, "bf16", 52)]
    lens = torch.tensor([50, 1, 2, 0, 30, 7], dtype=torch.int32, device="cuda")
    want = blk.attn_decode_shared(*args, lens)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = blk.attn_decode_shared(*args, lens)
        graphs.append((g, o))
    for _ in range(3):
        for g, o in graphs:
            o.zero_()
            g.replay()
            blk.attn_decode_shared(args[0].flip(0), *args[1:], lens)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for _, o in graphs)


def test_prefill_then_decode():
    """The two operators as a serving loop uses them: prompts prefilled behind
    a shared prefix, then one decode step over the prefix and the prompts' own
    caches is the prefill of the prompts with one token more."""
    H, Hk, d, P, dt = 8, 2, 128, 333, "bf16"
    lens = [40, 1, 129]
    longer = [n + 1 for n in lens]
    T = sum(longer)
    q, k, v = draw((H, T, d), dt, 61), draw((Hk, T, d), dt, 62), draw((Hk, T, d), dt, 63)
    kp, vp = draw((Hk, P, d), dt, 64), draw((Hk, P, d), dt, 65)
    cu = np.concatenate([[0], np.cumsum(longer)])
    qd, kd, vd, kpd, vpd = map(to_dev, (q, k, v, kp, vp))
    whole = blk.attn_prefill_packed(qd, kd, vd, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                    k_prefix=kpd, v_prefix=vpd)
    S = 200
    kc, vc = (torch.zeros((len(lens), Hk, S, d), dtype=kd.dtype, device="cuda") for _ in "kv")
    for b, n in enumerate(longer):
        kc[b, :, :n], vc[b, :, :n] = kd[:, cu[b]:cu[b + 1]], vd[:, cu[b]:cu[b + 1]]
    last = torch.from_numpy(cu[1:] - 1).cuda()
    o = blk.attn_decode_shared(qd[:, last].transpose(0, 1).contiguous(), kpd, vpd, kc, vc,
                               torch.tensor(longer, dtype=torch.int32, device="cuda"))
    # both within (u + 2^-14) sum p|v| + u |o| of the exact row; |o| <= sum p|v| <= max |v|
    bound = 2 * (2 * 2.0 ** -8 + 2.0 ** -14) * f64(v.abs().max())
    assert np.abs(f64(o) - f64(whole[last])).max() <= bound
    check(o, q[:, last.cpu()].transpose(0, 1), kp, vp, kc.cpu(), vc.cpu(), longer, dt, name="decode")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("H,Hk,d,keys", [(38, 19, 64, 768), (8, 1, 64, 61), (2, 2, 128, 384), (16, 4, 128, 200),
                                         (304, 304, 64, 30)])
def test_few_keys(dt, H, Hk, d, keys):
    """The kernel for few keys at its limits: batch 1 or more of many heads, a
    prefix of all keys but one, of none, and in between."""
    for B in (1, 3) if H <= 16 else (1,):
        for P in (0, 1, keys // 3, keys - 1):
            S = keys - P
            assert blk.attn_decode_shared_workspace_size(blk.decode_shared_desc(B, S, H, Hk, d, P)) == 0
            q, kp, vp, k, v = inputs(B, H, Hk, d, P, S, dt, 900 + P)
            lens = [S, 1, 0][:B]
            out = torch.full((B, H, d), 5.0, dtype=q.dtype, device="cuda")
            ref_slopes, dev_slopes = slopes_of(H, P % 2 == 0)
            blk.attn_decode_shared(*(None if t is None else to_dev(t) for t in (q, kp, vp, k, v)),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), alibi=P % 2 == 0,
                                   slopes=dev_slopes, out=out)
            check(out, q, kp, vp, k, v, lens, dt, ref_slopes, name=f"B {B} P {P}")


def test_binding_refuses():
    q, kp, vp, k, v = (to_dev(t) for t in inputs(2, 4, 2, 64, 32, 16, "bf16", 71))
    n = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        blk.attn_decode_shared(q, kp, None, k, v, n)
    with pytest.raises(ValueError):
        blk.attn_decode_shared(q, kp[:1], vp, k, v, n)
    with pytest.raises(ValueError):
        blk.attn_decode_shared(q, kp, vp, k[:1], v, n)
    with pytest.raises(ValueError):
        blk.attn_decode_shared(q, kp, vp, k, v, n[:1])
    with pytest.raises(TypeError):
        blk.attn_decode_shared(q, kp, vp, k, v, n.long())
    with pytest.raises(TypeError):
        blk.attn_decode_shared(q, kp.half(), vp, k, v, n)
    with pytest.raises(ValueError):
        blk.attn_decode_shared(q, kp.transpose(1, 2).contiguous().transpose(1, 2), vp, k, v, n)
    with pytest.raises(blk.BlkError):
        long = torch.zeros((2, 2, 16 + ROOM, 64), dtype=torch.bfloat16, device="cuda")
        blk.attn_decode_shared(q, kp, vp, long, long, n,
                               workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(blk.BlkError):
        blk.attn_decode_shared(q, kp, vp, k, v, n, slopes=torch.ones(4, device="cuda"))
