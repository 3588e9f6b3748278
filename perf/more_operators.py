"""The operators of a paged key/value cache: what a serving program calls for each chunk of a prompt and for each token.

``rope``: rotary positions of packed tokens at given positions: halves or interleaved pairs, a part of the head, scaled
for long contexts; queries and keys in one call.

``append``: the new tokens' keys (turned on the way) and values go into a paged cache, held in the storage type or in 8
bits (e4m3) with a scale for each page and head; the queries are turned along. One token for each sequence, or prompts.

``decode``: one decode step of attention over such a cache.

The 8-bit format: value = code * scale, where a page's scale (one for each key/value head, K and V apart) is the
smallest power of two of at least 2^-60 with which no code passes 448. It only grows while a page fills; the codes that
the page holds are then divided by the same power of two, and rounded.

Head shapes are those of this repository's configurations: Bloom-560m (16 x 64, ALiBi, fp16), StableLM-2-1.6B
(32 x 64, rotary over 16 of 64), OLMo-2-1B (16 x 128), StableLM-2-12B (32/8 x 160, rotary over 40 of 160) and the decode
benchmark's 32/8 x 128.
"""
import math
import random

import torch

own = False

HEADS = {  # query heads, key/value heads, head_dim, rotary span, rotary base
    "bloom": (16, 16, 64, 0, 10000.0),
    "stablelm": (32, 32, 64, 16, 10000.0),
    "olmo": (16, 16, 128, 128, 500000.0),
    "gqa128": (32, 8, 128, 128, 500000.0),
    "gqa160": (32, 8, 160, 40, 10000.0),
}
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
PAGES = (16, 32, 64, 128)
SCALING = ("none", "linear", "by_parts")
FACTOR, ORIGINAL, SLOW, FAST = 8.0, 8192, 1.0, 32.0  # of scaled positions: contexts 8 times those of training
LEAST, MOST = 2.0 ** -60, 448.0  # the least scale; the largest code


# ---------------------------------------------------------------- cases --
def rope(heads, dtype, tokens, far, interleaved, scaling):
    h, hk, d, span, base = HEADS[heads]
    return {"op": "rope", "heads": h, "kv_heads": hk, "head_dim": d, "span": span, "base": base, "dtype": dtype,
            "tokens": tokens, "far": far, "interleaved": interleaved, "scaling": scaling}


def append(heads, dtype, bits, page, batch, new, before, interleaved, scaling, ragged):
    h, hk, d, span, base = HEADS[heads]
    return {"op": "append", "heads": h, "kv_heads": hk, "head_dim": d, "span": span, "base": base, "dtype": dtype,
            "bits": bits, "page": page, "batch": batch, "new": new, "before": before, "interleaved": interleaved,
            "scaling": scaling, "ragged": ragged}


def decode(heads, dtype, bits, page, batch, longest, alibi, ragged):
    h, hk, d, _, _ = HEADS[heads]
    return {"op": "decode", "heads": h, "kv_heads": hk, "head_dim": d, "dtype": dtype, "bits": bits, "page": page,
            "batch": batch, "longest": longest, "alibi": alibi, "ragged": ragged}


def listed():
    return [
        # the newest tokens of 24 users: latency
        dict(rope("olmo", "bf16", 24, 8000, False, "none"), name="rope step, 16 x 128"),
        # a batch of prompts, a quarter of each head turned
        dict(rope("stablelm", "bf16", 4093, 4096, False, "none"), name="rope prompts, 16 of 64"),
        # long documents with scaled positions, interleaved pairs
        dict(rope("gqa128", "fp16", 16384, 65536, True, "by_parts"), name="rope documents, scaled"),
        # a decode step of 16 users: latency
        dict(append("gqa128", "bf16", 8, 16, 16, 1, 4000, False, "none", 1), name="append step, 8 bits"),
        # ordinary chunks of prompts, some of which go on in a page that is part full
        dict(append("stablelm", "bf16", 8, 32, 6, 1500, 700, False, "none", 2), name="append prompts, 8 bits"),
        # the same in the storage type, without a rotary
        dict(append("bloom", "fp16", 16, 16, 12, 901, 300, False, "none", 3), name="append prompts, 16 bits"),
        # a large prefill
        dict(append("gqa128", "bf16", 8, 64, 32, 2047, 2000, True, "linear", 4), name="append large, 8 bits"),
        # a few users with short contexts: latency
        dict(decode("bloom", "fp16", 8, 16, 4, 500, True, 5), name="decode small, bloom"),
        # a chat service
        dict(decode("gqa128", "bf16", 8, 64, 32, 4099, False, 6), name="decode chat, 32/8 x 128"),
        # the wide heads of the 12B model
        dict(decode("gqa160", "bf16", 8, 32, 24, 6001, False, 7), name="decode chat, 32/8 x 160"),
        # a few long documents in a cache of the storage type
        dict(decode("olmo", "bf16", 16, 64, 8, 32771, False, 8), name="decode documents, 16 bits"),
        # many users, from a few tokens to 16k
        dict(decode("gqa128", "fp16", 8, 64, 96, 16384, False, 9), name="decode large, 32/8 x 128"),
    ]


def spread(rng, lo, hi):
    """A whole number in [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {op: [c for c in listed() if c["op"] == op] for op in ("rope", "append", "decode")}
    while True:
        op, heads, dtype = rng.choice(sorted(most)), rng.choice(sorted(HEADS)), rng.choice(sorted(DTYPES))
        bits, page, ragged = rng.choice((8, 8, 16)), rng.choice(PAGES), rng.randrange(1000, 1 << 20)
        interleaved, scaling = rng.random() < 0.5, rng.choice(SCALING)
        if op == "rope":
            if heads == "bloom":  # ALiBi: nothing to turn
                continue
            c = rope(heads, dtype, spread(rng, 1, 16384), spread(rng, 100, 1 << 20), interleaved, scaling)
        elif op == "append":
            new = 1 if rng.random() < 0.4 else spread(rng, 2, 4096)
            c = append(heads, dtype, bits, page, spread(rng, 1, 256), new, spread(rng, 1, 16384), interleaved, scaling,
                       ragged)
            if sum(pages_of(c)) * page > 1 << 19:
                continue
        else:
            c = decode(heads, dtype, bits, page, spread(rng, 1, 256), spread(rng, 16, 65536), rng.random() < 0.3, ragged)
            if c["batch"] * c["longest"] * c["kv_heads"] * c["head_dim"] > 96 * 16384 * 8 * 128:
                continue
        top = max(work(x)["bytes"] for x in most[op])
        if work(c)["bytes"] <= top:
            return c


def counts(case):
    """(tokens in the cache before, new tokens) of each sequence: the longest at a drawn place, the others spread."""
    r = random.Random(case["ragged"])
    n = case["batch"]
    if case["op"] == "decode":
        new = [0] * n
        before = [spread(r, max(1, case["longest"] // 16), case["longest"]) for _ in range(n)]
        before[r.randrange(n)] = case["longest"]
    elif case["new"] == 1:
        new = [1] * n
        before = [r.randint(0, case["before"]) for _ in range(n)]
    else:
        new = [spread(r, max(1, case["new"] // 8), case["new"]) for _ in range(n)]
        new[r.randrange(n)] = case["new"]
        before = [r.randint(1, case["before"]) if r.random() < 0.3 else 0 for _ in range(n)]
    return before, new


def pages_of(case):
    """Pages of each sequence, with its new tokens."""
    before, new = counts(case)
    return [-(-(b + n) // case["page"]) for b, n in zip(before, new)]


def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rope":
        n = case["tokens"]
        return {"bytes": 4 * n * (h + hk) * d + 4 * n, "flops": 3 * n * (h + hk) * case["span"]}
    before, new = counts(case)
    wide = case["bits"] // 8
    if case["op"] == "append":
        t = sum(new)
        touched = sum((b + n - 1) // case["page"] - b // case["page"] + 1 for b, n in zip(before, new))
        scales = 2 * 4 * touched * hk if wide == 1 else 0
        turned = 4 * t * h * d if case["span"] else 0
        return {"bytes": t * hk * d * (4 + 2 * wide) + turned + scales + 4 * touched + 8 * len(new),
                "flops": 3 * t * (h + hk) * case["span"] + (4 * t * hk * d if wide == 1 else 0)}
    t, p = sum(before), sum(pages_of(case))
    return {"bytes": 2 * t * hk * d * wide + (2 * 4 * p * hk if wide == 1 else 0) + 4 * p
            + 4 * len(before) * h * d + 4 * len(before), "flops": 4 * t * h * d}


# --------------------------------------------------------------- inputs --
def frequencies(case):
    """Radians per position of each pair, in 64 bits, and the amplitude of the turned part."""
    if case["scaling"] == "none" or not case["span"]:
        factor = 1.0
    else:
        factor = FACTOR
    theta = torch.pow(torch.tensor(case["base"], dtype=torch.float64),
                      -2.0 * torch.arange(case["span"] // 2, dtype=torch.float64) / max(1, case["span"]))
    if case["scaling"] == "by_parts":
        keep = ((theta * ORIGINAL / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0.0, 1.0)
        return (theta * (keep + (1.0 - keep) / factor)).cuda(), 0.1 * math.log(factor) + 1.0
    return (theta / factor).cuda(), 1.0


def plan_of(case):
    """The plan that a user's program makes once for a model."""
    if not own or not case["span"]:
        return None
    import alibi_attention_block_gb300 as blk
    kind = case["scaling"]
    more = {} if kind == "none" else {"scaling": kind, "factor": FACTOR}
    if kind == "by_parts":
        more.update(original_len=ORIGINAL, beta_slow=SLOW, beta_fast=FAST, amplitude=0.1 * math.log(FACTOR) + 1.0)
    return blk.rope_plan(case["span"], case["base"], interleaved=case["interleaved"], **more)


def tables(case, g):
    """A block table whose pages lie anywhere in the pool, -1 behind a sequence's last, and the pool's pages."""
    n = pages_of(case)
    pool = sum(n) + 3
    place = torch.randperm(pool, generator=g, device="cuda")[:sum(n)].to(torch.int32)
    count = torch.tensor(n, device="cuda")
    column = torch.arange(max(n), device="cuda")
    table = torch.full((len(n), max(n)), -1, dtype=torch.int32, device="cuda")
    table[column < count[:, None]] = place
    return table, pool


def held(x, bits, dt):
    """x [pages, kv heads, tokens, d] as a cache holds it: (codes or values, scales or None)."""
    if bits == 16:
        return x.to(dt), None
    scale = page_scale(x.abs().amax((2, 3)).float())
    return (x / scale[:, :, None, None].to(x.dtype)).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    h, hk, d, dt = case["heads"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + case.get("ragged", case.get("tokens", 0)))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    # keys as a projection with a bias gives them: a part that all tokens of a head share, and each token's own
    k_mean, v_mean = 0.5 * normal(hk, 1, d), 0.5 * normal(hk, 1, d)
    s = {"case": case}
    if case["op"] == "rope":
        n = case["tokens"]
        s["q"], s["k"] = normal(h, n, d).to(dt), (normal(hk, n, d) + k_mean).to(dt)
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["turn"], s["plan"] = frequencies(case), plan_of(case)
        return s
    before, new = counts(case)
    s["table"], pool = tables(case, g)
    s["lens"] = torch.tensor([b + n for b, n in zip(before, new)], dtype=torch.int32, device="cuda")
    for name, mean in (("k", k_mean), ("v", v_mean)):
        x = normal(pool, hk, case["page"], d, dtype=torch.bfloat16) + mean.bfloat16()
        s[name + "_cache"], s[name + "_scale"] = held(x, case["bits"], dt)
    if case["op"] == "decode":
        s["q"] = normal(len(before), h, d).to(dt)
        return s
    t, ends = sum(new), [0]
    for n in new:
        ends.append(ends[-1] + n)
    s["cu_seqlens"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    s["q"] = normal(h, t, d).to(dt) if case["span"] else None
    loud = 1.0 + 3.0 * (torch.rand((1, t, 1), generator=g, device="cuda") < 0.02)  # some tokens stand out
    s["k"], s["v"] = (normal(hk, t, d) * loud + k_mean).to(dt), (normal(hk, t, d) + v_mean).to(dt)
    s["turn"], s["plan"] = frequencies(case), plan_of(case)
    return s


# ---------------------------------------------------------- plain forms --
def page_scale(amax):
    """The smallest power of two of at least LEAST with which amax takes a code of at most MOST."""
    mantissa, exponent = torch.frexp(amax)  # in [0.5, 1); MOST is 0.875 * 2^9
    scale = torch.ldexp(torch.ones_like(amax), exponent - 9 + (mantissa > MOST / 512).to(exponent.dtype))
    return torch.where(amax > 0, scale, 0.0).clamp_min(LEAST)


def plain_turn(x, positions, case, theta, amplitude):
    """x [n, T, d] turned at its tokens' positions, in 32 bits (the angles in 64)."""
    span, x = case["span"], x.float()
    if not span:
        return x
    angle = positions.double()[:, None] * theta
    cos, sin = (amplitude * angle.cos()).float(), (amplitude * angle.sin()).float()
    part = x[..., :span]
    if case["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :span // 2], part[..., span // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., span:]), -1)


def plain_rope(s):
    return [plain_turn(s[n], s["positions"], s["case"], *s["turn"]).to(s[n].dtype) for n in ("q", "k")]


def plain_append(s):
    case, table, lens, cu = s["case"], s["table"], s["lens"].long(), s["cu_seqlens"].long()
    page, new = case["page"], cu[1:] - cu[:-1]
    t = s["k"].shape[1]
    token = torch.arange(t, device=table.device)
    of = torch.bucketize(token, cu[1:], right=True)  # the token's sequence
    position = lens[of] - cu[of + 1] + token
    where, offset = table[of, position // page].long(), position % page
    first = lens - new  # the sequences' first new positions, and those positions' pages
    head = table[torch.arange(len(lens), device=table.device), first // page].long()
    goes_on = first % page > 0
    for name in ("k", "v"):  # the two caches
        cache, scale, dt = s[name + "_cache"], s[name + "_scale"], s[name].dtype
        x = plain_turn(s[name], position, case, *s["turn"]) if name == "k" else s[name].float()
        if scale is None:
            cache[where, :, offset] = x.to(dt).transpose(0, 1)
            continue
        amax = torch.zeros_like(scale).index_reduce_(0, where, x.abs().amax(-1).t(), "amax")
        last = scale[head]
        fresh = page_scale(amax)
        grown = torch.where(goes_on[:, None], torch.maximum(fresh[head], last), fresh[head])
        scale[where] = fresh[where]
        scale[head] = grown
        # what the part-full pages hold, at the grown scale
        codes = cache.view(torch.uint8)
        old = codes[head].view(torch.float8_e4m3fn).float() * (last / grown)[:, :, None, None]
        mine = torch.arange(page, device=table.device) < (first % page)[:, None]
        codes[head] = torch.where(mine[:, None, :, None], old.to(torch.float8_e4m3fn).view(torch.uint8), codes[head])
        fits = x.transpose(0, 1) / scale[where][..., None]
        codes[where, :, offset] = fits.to(torch.float8_e4m3fn).view(torch.uint8)
    turned = None if s["q"] is None else plain_turn(s["q"], position, case, *s["turn"]).to(s["q"].dtype)
    return appended(s, turned)


def appended(s, q):
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def plain_held(cache, scale, table):
    """Each sequence's keys or values in 32 bits: [b, hk, capacity, d]."""
    at = table.clamp_min(0).long()
    if scale is None:
        x = cache[at].float()
    else:
        x = cache.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][..., None, None]
    b, p, hk, n, d = x.shape
    return x.transpose(1, 2).reshape(b, hk, p * n, d)


def plain_decode(s):
    q, lens = s["q"], s["lens"].long()
    b, h, d = q.shape
    k = plain_held(s["k_cache"], s["k_scale"], s["table"])
    hk, n = k.shape[1], k.shape[2]
    scores = torch.matmul(q.float().view(b, hk, h // hk, d) * d ** -0.5, k.transpose(-1, -2))
    del k
    far = torch.arange(n, device=q.device) - (lens - 1)[:, None]  # key position - query position
    if s["case"]["alibi"]:
        slopes = torch.exp2(-8.0 * torch.arange(1, h + 1, device=q.device, dtype=torch.float32) / h)
        scores += slopes.view(hk, h // hk, 1) * far[:, None, None]
    scores.masked_fill_((far > 0)[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    scores /= scores.sum(-1, keepdim=True)
    return torch.matmul(scores, plain_held(s["v_cache"], s["v_scale"], s["table"])).reshape(b, h, d).to(q.dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        import alibi_attention_block_gb300 as blk
        if op == "rope":
            return blk.rope_positions(s["q"], s["positions"], s["plan"], k=s["k"])
        if op == "append":
            return appended(s, blk.kv_append_paged(
                s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], cu_seqlens=s["cu_seqlens"],
                k_scale=s["k_scale"], v_scale=s["v_scale"], rope=s["plan"], q=s["q"]))
        return blk.attn_decode_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], k_scale=s["k_scale"],
                                     v_scale=s["v_scale"], alibi=s["case"]["alibi"])
    return plain_rope(s) if op == "rope" else plain_append(s) if op == "append" else plain_decode(s)


# -------------------------------------------------------- in 64 bits -----
def exact_turn(x, positions, case):
    """Each pair as a complex number, times amplitude * e^(i angle)."""
    span, out = case["span"], x.double().clone()
    for j in range(span // 2):
        theta = case["base"] ** (-2.0 * j / span)
        size = 1.0
        if case["scaling"] == "linear":
            theta /= FACTOR
        elif case["scaling"] == "by_parts":
            turns = ORIGINAL * theta / (2 * math.pi)
            part = min(1.0, max(0.0, (turns - SLOW) / (FAST - SLOW)))
            theta = part * theta + (1 - part) * theta / FACTOR
            size = 1 + 0.1 * math.log(FACTOR)
        first, second = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + span // 2)
        turn = torch.polar(torch.full_like(positions, size, dtype=torch.float64), positions.double() * theta)
        z = torch.complex(x[..., first].double(), x[..., second].double()) * turn
        out[..., first], out[..., second] = z.real, z.imag
    return out


def exact_code(x):
    """The nearest e4m3 number, ties to even: three bits behind the leading one, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact_scale(amax):
    return 2.0 ** max(-60, math.ceil(math.log2(amax / 448.0))) if amax > 0 else 2.0 ** -60


def exact_append(s, case):
    before, new = counts(case)
    table, start, page, position = s["table"].tolist(), 0, case["page"], []
    for b, n in zip(before, new):
        position += range(b, b + n)
    position = torch.tensor(position, device="cuda")
    out = {"q": None if s["q"] is None else exact_turn(s["q"], position, case)}
    x = {"k": exact_turn(s["k"], position, case), "v": s["v"].double()}
    for name in ("k", "v"):
        cache = s[name + "_cache"].double()
        scale = None if s[name + "_scale"] is None else s[name + "_scale"].double().cpu()
        rows, starts, places = x[name], [], []
        if scale is not None:
            largest = rows.abs().amax(-1).cpu()
            scaled = torch.ones(rows.shape[:2], dtype=torch.float64)
        start = 0
        for i, (b, n) in enumerate(zip(before, new)):
            at = 0
            while at < n:
                place, offset = table[i][(b + at) // page], (b + at) % page
                m = min(page - offset, n - at)
                places.append((place, offset, m))
                starts.append(start + at)
                if scale is not None:
                    top = largest[:, start + at:start + at + m].amax(-1).tolist()
                    for head in range(len(top)):
                        want = exact_scale(top[head])
                        if offset:
                            was = float(scale[place, head])
                            want = max(want, was)
                            if want > was:
                                cache[place, head, :offset] = exact_code(cache[place, head, :offset] * (was / want))
                        scale[place, head] = want
                        scaled[head, start + at:start + at + m] = want
                at += m
            start += n
        if scale is not None:
            rows = exact_code(rows / scaled.to(rows.device)[..., None])
        for at, (place, offset, m) in zip(starts, places):
            cache[place, :, offset:offset + m] = rows[:, at:at + m]
        out[name], out[name + "_scale"] = cache, None if scale is None else scale.cuda()
    return out


def exact_decode(s, case):
    q, page, lens = s["q"], case["page"], counts(case)[0]
    b, h, d = q.shape
    hk = case["kv_heads"]
    grp = h // hk
    out = torch.empty((b, h, d), dtype=torch.float64, device=q.device)
    for i, n in enumerate(lens):
        places = s["table"][i, :-(-n // page)].long()

        def whole(name):
            x = s[name + "_cache"].view(torch.uint8 if case["bits"] == 8 else q.dtype)[places]
            if case["bits"] == 8:
                x = x.view(torch.float8_e4m3fn).double() * s[name + "_scale"][places].double()[..., None, None]
            return x.double().permute(1, 0, 2, 3).reshape(hk, -1, d)[:, :n]

        logits = torch.einsum("kgd,knd->kgn", q[i].double().view(hk, grp, d), whole("k")) / math.sqrt(d)
        if case["alibi"]:
            slope = torch.tensor([2.0 ** (-8.0 * (j + 1) / h) for j in range(h)], dtype=torch.float64, device=q.device)
            logits = logits - slope.view(hk, grp, 1) * torch.arange(n - 1, -1, -1, device=q.device)
        out[i] = torch.einsum("kgn,knd->kgd", torch.softmax(logits, -1), whole("v")).reshape(h, d)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return [exact_turn(s[n], s["positions"], case) for n in ("q", "k")]
    return exact_append(s, case) if case["op"] == "append" else exact_decode(s, case)
