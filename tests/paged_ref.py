"""The paged cache's operators from their definitions, in 64 bits (NumPy): what the GPU
tests compare with. Steps of a type: u = eps / 2 relative, half of one."""
import math

import numpy as np
import torch

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def thetas(span, base=10000.0, scaling="none", factor=1.0, original_len=0.0, beta_slow=1.0, beta_fast=32.0):
    """Radians per position of each pair."""
    out = []
    for j in range(span // 2):
        th = base ** (-2.0 * j / span)
        if scaling == "linear":
            th /= factor
        elif scaling == "by_parts":
            turns = original_len * th / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)))
            th = g * th + (1 - g) * th / factor
        out.append(th)
    return np.array(out)


def turn(x, positions, th, interleaved, amplitude=1.0, inverse=False):
    """x [n, T, d] -> (turned, sum of the magnitudes that make up each value)."""
    x = np.asarray(x, dtype=np.float64)
    y, mag = x.copy(), np.abs(x)
    for j, t in enumerate(th):
        i, k = (2 * j, 2 * j + 1) if interleaved else (j, j + len(th))
        a = np.asarray(positions, dtype=np.float64) * t * (-1 if inverse else 1)
        c, s = amplitude * np.cos(a), amplitude * np.sin(a)
        y[..., i], y[..., k] = x[..., i] * c - x[..., k] * s, x[..., k] * c + x[..., i] * s
        mag[..., i] = mag[..., k] = amplitude * (np.abs(x[..., i]) + np.abs(x[..., k]))
    return y, mag


def e4m3(x):
    """The nearest e4m3 number, ties to even, at most 448."""
    a = np.minimum(np.abs(x), 448.0)
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.sign(x) * np.round(a / step) * step


def page_scale(most):
    return 2.0 ** max(-60, math.ceil(math.log2(most / 448.0))) if most > 0 else 2.0 ** -60


def values(cache, scale):
    """A cache [pages, Hk, n, d] as the numbers it stands for."""
    x = cache.cpu().float().double().numpy()
    return x if scale is None else x * scale.cpu().double().numpy()[..., None, None]


def rows(cache, scale, table, n, page):
    """The first n positions of a sequence: ([Hk, n, d], seen [n], scale [Hk, n])."""
    at = torch.as_tensor(table[:-(-n // page)], dtype=torch.long, device=cache.device)
    ok = (at >= 0) & (at < cache.shape[0])
    x = cache[at.clamp(0, cache.shape[0] - 1)].float().double()
    s = torch.ones(x.shape[:2], dtype=torch.float64, device=x.device)
    if scale is not None:
        s = scale[at.clamp(0, cache.shape[0] - 1)].double()
        x = x * s[..., None, None]
    x = x.transpose(0, 1).flatten(1, 2)[:, :n].cpu().numpy()
    seen = ok.repeat_interleave(page)[:n].cpu().numpy()
    return np.where(seen[None, :, None], x, 0.0), seen, s.t().repeat_interleave(page, 1)[:, :n].cpu().numpy()


def decode(q, k, v, seen, slopes=None, scale=None):
    """q [H, d], k and v [Hk, n, d] -> (o, sum p |v|, p [H, n])."""
    H, d = q.shape
    grp = H // k.shape[0]
    kk, vv = np.repeat(k, grp, 0), np.repeat(v, grp, 0)
    n = k.shape[1]
    s = np.einsum("hd,hnd->hn", q, kk) * (d ** -0.5 if scale is None else scale)
    if slopes is not None:
        s = s - np.asarray(slopes)[:, None] * (n - 1 - np.arange(n))
    s = np.where(seen, s, -np.inf)
    if not seen.any():
        z = np.zeros((H, d))
        return z, z, np.zeros((H, n))
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    vv = np.where(seen[:, None], vv, 0.0)
    return np.einsum("hn,hnd->hd", p, vv), np.einsum("hn,hnd->hd", p, np.abs(vv)), p
