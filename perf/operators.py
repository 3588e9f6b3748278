"""Attention over packed prompts and over a prefix that a batch shares: the calls a serving program makes.

``packed``: causal attention over several prompts of different lengths that lie one behind the other in
one token axis (``cu_seqlens``), with grouped heads, optionally ALiBi, optionally behind a prefix of keys that every
prompt shares (a common system prompt whose keys and values exist already).

``shared``: one decode step of a batch whose sequences share a long prefix: each sequence's newest token attends
to the prefix (stored once) and to the sequence's own cache.

Head shapes are those of this repository's configurations: Bloom-560m (16 x 64, ALiBi, fp16), StableLM-2-1.6B
(32 x 64), OLMo-2-1B (16 x 128), StableLM-2-12B (32/8 x 160) and the decode benchmark's 32/8 x 128.
"""
import math
import random

import torch

own = False

HEADS = {  # query heads, key/value heads, head_dim
    "bloom": (16, 16, 64),
    "stablelm": (32, 32, 64),
    "olmo": (16, 16, 128),
    "gqa128": (32, 8, 128),
    "gqa160": (32, 8, 160),
}
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases --
def packed(heads, dtype, alibi, prompts, longest, prefix, ragged):
    h, hk, d = HEADS[heads]
    return {"op": "packed", "heads": h, "kv_heads": hk, "head_dim": d, "dtype": dtype, "alibi": alibi,
            "prompts": prompts, "longest": longest, "prefix": prefix, "ragged": ragged}


def shared(heads, dtype, alibi, batch, prefix, capacity, ragged):
    h, hk, d = HEADS[heads]
    return {"op": "shared", "heads": h, "kv_heads": hk, "head_dim": d, "dtype": dtype, "alibi": alibi,
            "batch": batch, "prefix": prefix, "capacity": capacity, "ragged": ragged}


def listed():
    return [
        # sixteen short chat turns in one pass: the launch and each item's latency count
        dict(packed("bloom", "fp16", True, 16, 61, 0, 1), name="packed chat turns, bloom"),
        # an ordinary prefill batch of a serving loop, about 8000 tokens
        dict(packed("stablelm", "bf16", False, 8, 2047, 0, 2), name="packed prefill, 32 x 64"),
        # the same with wide heads: documents of a few thousand tokens
        dict(packed("olmo", "bf16", False, 5, 3500, 0, 3), name="packed documents, 16 x 128"),
        # grouped heads of the 12B model, head_dim 160
        dict(packed("gqa160", "bf16", False, 6, 2000, 0, 4), name="packed prefill, 32/8 x 160"),
        # many short user prompts behind one system prompt
        dict(packed("gqa128", "bf16", False, 32, 300, 2000, 5), name="packed behind a prefix, 32/8 x 128"),
        # long documents
        dict(packed("stablelm", "bf16", False, 2, 8192, 0, 6), name="packed long, 32 x 64"),
        # a few users on a short system prompt: latency
        dict(shared("bloom", "fp16", True, 4, 500, 64, 7), name="shared small, bloom"),
        # a chat service: 32 users on an 8k system prompt
        dict(shared("stablelm", "bf16", False, 32, 8192, 512, 8), name="shared chat, 32 x 64"),
        # grouped heads, long prefix, long own caches
        dict(shared("gqa128", "bf16", False, 64, 16384, 1024, 9), name="shared long, 32/8 x 128"),
        # a wide batch: the products with the prefix no longer hide behind its bytes
        dict(shared("gqa128", "bf16", False, 256, 4099, 200, 10), name="shared wide, 32/8 x 128"),
        # questions about one document of 32k tokens
        dict(shared("olmo", "fp16", False, 16, 32771, 2048, 11), name="shared document, 16 x 128"),
        # ALiBi over a long prefix
        dict(shared("bloom", "fp16", True, 24, 20000, 700, 12), name="shared alibi, bloom"),
    ]


def spread(rng, lo, hi):
    """A whole number in [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def padded(c):
    """Score elements of the padded plain form of a packed case."""
    return c["prompts"] * c["heads"] * c["longest"] * (c["longest"] + c["prefix"])


def draw(rng):
    most = {op: [c for c in listed() if c["op"] == op] for op in ("packed", "shared")}
    while True:
        heads, dtype, ragged = rng.choice(sorted(HEADS)), rng.choice(sorted(DTYPES)), rng.randrange(1000, 1 << 20)
        alibi = rng.random() < 0.3
        if rng.random() < 0.5:
            prefix = spread(rng, 1, 4096) if rng.random() < 0.4 else 0
            c = packed(heads, dtype, alibi, spread(rng, 1, 64), spread(rng, 16, 8192), prefix, ragged)
            if padded(c) > max(padded(x) for x in most["packed"]):
                continue
        else:
            if heads == "gqa160":  # the framework's decode step has head_dim 64 and 128
                continue
            c = shared(heads, dtype, alibi, spread(rng, 1, 256), spread(rng, 64, 32768), spread(rng, 1, 2048), ragged)
        top = {k: max(work(x)[k] for x in most[c["op"]]) for k in ("bytes", "flops")}
        if all(work(c)[k] <= top[k] for k in top):
            return c


def lengths(case):
    """Tokens of each prompt, or of each sequence's own cache: the longest at a drawn place, the others spread."""
    r = random.Random(case["ragged"])
    if case["op"] == "packed":
        n = [spread(r, max(1, case["longest"] // 8), case["longest"]) for _ in range(case["prompts"])]
        n[r.randrange(len(n))] = case["longest"]
    else:
        n = [r.randint(1, case["capacity"]) for _ in range(case["batch"])]
        n[r.randrange(len(n))] = case["capacity"]
    return n


def work(case):
    h, hk, d, p, n = case["heads"], case["kv_heads"], case["head_dim"], case["prefix"], lengths(case)
    t = sum(n)
    if case["op"] == "packed":
        pairs = sum(m * (m + 1) // 2 + m * p for m in n)
        elements = 2 * t * h * d + 2 * (t + p) * hk * d  # q and o; k and v with the prefix's
    else:
        pairs = sum(p + m for m in n)
        elements = 2 * len(n) * h * d + 2 * (t + p) * hk * d
    return {"bytes": 2 * elements + 4 * (len(n) + 1), "flops": 4 * d * h * pairs}


# --------------------------------------------------------------- inputs --
def prepare(case, seed):
    h, hk, d, p = case["heads"], case["kv_heads"], case["head_dim"], case["prefix"]
    dt, n = DTYPES[case["dtype"]], lengths(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + case["ragged"])

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    # a projection with a bias: a part that all tokens of a head share, and each token's own
    k_mean, v_mean = 0.5 * normal(hk, 1, d), 0.5 * normal(hk, 1, d)
    s = {"op": case["op"], "alibi": case["alibi"], "prefix": p, "longest": max(n),
         "k_prefix": (normal(hk, p, d) + k_mean).to(dt) if p else None,
         "v_prefix": (normal(hk, p, d) + v_mean).to(dt) if p else None}
    if case["op"] == "packed":
        t, ends = sum(n), [0]
        for m in n:
            ends.append(ends[-1] + m)
        s["q"] = normal(h, t, d).to(dt)
        s["k"], s["v"] = (normal(hk, t, d) + k_mean).to(dt), (normal(hk, t, d) + v_mean).to(dt)
        s["cu_seqlens"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    else:
        b, c = case["batch"], case["capacity"]
        s["q"] = normal(b, h, d).to(dt)
        s["k"], s["v"] = (normal(b, hk, c, d) + k_mean).to(dt), (normal(b, hk, c, d) + v_mean).to(dt)
        s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------- plain forms --
def plain_softmax(scores):
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    scores /= scores.sum(-1, keepdim=True)
    return scores


def plain_slopes(h, device):
    return torch.exp2(-8.0 * torch.arange(1, h + 1, device=device, dtype=torch.float32) / h)


def plain_packed(s):
    """The prompts padded to the longest; scores of every query with the prefix's keys and its own prompt's."""
    q, k, v, cu, p, n = s["q"], s["k"], s["v"], s["cu_seqlens"], s["prefix"], s["longest"]
    h, t, d = q.shape
    hk, b = k.shape[0], cu.numel() - 1
    grp = h // hk
    step = torch.arange(n, device=q.device)
    inside = step < (cu[1:] - cu[:-1])[:, None]
    rows = torch.where(inside, cu[:-1, None] + step, 0)  # [b, n]: the packed row of each padded place
    qp = q.float()[:, rows].view(hk, grp, b, n, d).permute(2, 0, 1, 3, 4).reshape(b, hk, grp * n, d)
    kp, vp = k.float()[:, rows].transpose(0, 1), v.float()[:, rows].transpose(0, 1)  # [b, hk, n, d]
    if p:
        kp = torch.cat([s["k_prefix"].float().expand(b, hk, p, d), kp], 2)
        vp = torch.cat([s["v_prefix"].float().expand(b, hk, p, d), vp], 2)
    scores = torch.matmul(qp * d ** -0.5, kp.transpose(-1, -2)).view(b, hk, grp, n, p + n)
    far = torch.arange(p + n, device=q.device) - (p + step)[:, None]  # key position - query position
    if s["alibi"]:
        scores += plain_slopes(h, q.device).view(hk, grp, 1, 1) * far
    scores.masked_fill_(far > 0, -math.inf)
    o = torch.matmul(plain_softmax(scores).view(b, hk, grp * n, p + n), vp).view(b, h, n, d)
    token = torch.arange(t, device=q.device)
    which = (token[:, None] >= cu[1:]).sum(1)
    return o[which, :, token - cu[which]].to(q.dtype)


def plain_shared(s):
    """Scores of each newest token with the prefix's keys (one product for the batch) and its own cache's."""
    q, kc, vc, lens, p = s["q"], s["k"], s["v"], s["lens"], s["prefix"]
    b, h, d = q.shape
    hk, c = kc.shape[1], kc.shape[2]
    grp = h // hk
    qf = q.float().view(b, hk, grp, d) * d ** -0.5
    kp, vp = s["k_prefix"].float(), s["v_prefix"].float()
    ahead = torch.matmul(qf.transpose(0, 1).reshape(hk, b * grp, d), kp.transpose(-1, -2))
    ahead = ahead.view(hk, b, grp, p).transpose(0, 1)
    scores = torch.cat([ahead, torch.matmul(qf, kc.float().transpose(-1, -2))], -1)  # [b, hk, grp, p + c]
    far = torch.arange(p + c, device=q.device) - (p + lens[:, None] - 1)
    if s["alibi"]:
        scores += plain_slopes(h, q.device).view(hk, grp, 1) * far[:, None, None]
    scores.masked_fill_((far > 0)[:, None, None], -math.inf)
    w = plain_softmax(scores)
    o = torch.matmul(w[..., :p].transpose(0, 1).reshape(hk, b * grp, p), vp).view(hk, b, grp, d).transpose(0, 1)
    return (o + torch.matmul(w[..., p:], vc.float())).reshape(b, h, d).to(q.dtype)


def run(s):
    if own:
        import alibi_attention_block_gb300 as blk
        if s["op"] == "packed":
            return blk.attn_prefill_packed(s["q"], s["k"], s["v"], s["cu_seqlens"], k_prefix=s["k_prefix"],
                                           v_prefix=s["v_prefix"], alibi=s["alibi"])
        return blk.attn_decode_shared(s["q"], s["k_prefix"], s["v_prefix"], s["k"], s["v"], s["lens"],
                                      alibi=s["alibi"])
    return plain_packed(s) if s["op"] == "packed" else plain_shared(s)


# -------------------------------------------------------- in 64 bits -----
def attend(q, k, v, first, slopes):
    """softmax(q k^T / sqrt(d) + bias) v of one kv head in 64 bits: q [grp, m, d] at positions first.., k, v [n, d]."""
    grp, m, d = q.shape
    logits = torch.einsum("gmd,nd->gmn", q.double(), k.double()) / math.sqrt(d)
    query = torch.arange(first, first + m, device=q.device).view(m, 1)
    key = torch.arange(k.shape[0], device=q.device).view(1, -1)
    if slopes is not None:
        logits = logits - slopes.view(-1, 1, 1) * (query - key)
    logits = logits.masked_fill(key > query, -math.inf)
    return torch.einsum("gmn,nd->gmd", torch.softmax(logits, -1), v.double())


def exact(case, seed):
    s = prepare(case, seed)
    h, hk, d, p, n = case["heads"], case["kv_heads"], case["head_dim"], case["prefix"], lengths(case)
    if 4 * d * h * sum(m * (m + p) for m in n) > 4e12 and case["op"] == "packed":
        return None
    grp, dev = h // hk, s["q"].device
    slopes = [2.0 ** (-8.0 * (i + 1) / h) for i in range(h)]
    slopes = torch.tensor(slopes, dtype=torch.float64, device=dev) if case["alibi"] else None
    at = 0
    out = torch.empty((sum(n) if case["op"] == "packed" else len(n), h, d), dtype=torch.float64, device=dev)
    for b, m in enumerate(n):
        for i in range(hk):
            mine = slice(i * grp, (i + 1) * grp)
            if case["op"] == "packed":
                q, k, v = s["q"][mine, at:at + m], s["k"][i, at:at + m], s["v"][i, at:at + m]
                first = p
            else:
                q, k, v = s["q"][b, mine].unsqueeze(1), s["k"][b, i, :m], s["v"][b, i, :m]
                first = p + m - 1
            if p:
                k, v = torch.cat([s["k_prefix"][i], k]), torch.cat([s["v_prefix"][i], v])
            o = attend(q, k, v, first, None if slopes is None else slopes[mine])
            if case["op"] == "packed":
                out[at:at + m, mine] = o.transpose(0, 1)
            else:
                out[b, mine] = o[:, 0]
        at += m
    return out
