"""Plain float64 forms of the serving-step operators (torch, CPU or GPU), for the tests of
kvc_append_qk, kvc_decode_attention_scored, kvc_prefill_scored and kvc_decode_attention_shared."""

from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def frequencies(dim, base=10000.0, scaling="none", factor=1.0, original_len=0, fast=32.0, slow=1.0):
    """Angle for each position step of pair i = 0 .. dim / 2 - 1 (list of floats), and the magnitude."""
    out, mag = [], 1.0
    low = high = 0.0
    if scaling == "yarn" and dim:
        def pair_of(turns):
            return dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), dim - 1)
        if factor > 1:
            mag = 0.1 * math.log(factor) + 1.0
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            f = f / factor * r + f * (1 - r)
        elif scaling == "bands":
            r = min(max((original_len * f / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0)
            f = f / factor * (1 - r) + f * r
        out.append(f)
    return out, mag


def norm(x, w, eps, offset):
    if w is None:
        return x
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * (w.double() + offset)


def rotate(x, pos, freq, mag, pairs):
    """x [..., heads, D] float64 at positions pos [...]: rotated in the first 2 * len(freq) values."""
    n = 2 * len(freq)
    if n == 0:
        return x
    f = torch.tensor(freq, dtype=torch.float64, device=x.device)
    ang = (pos.double()[..., None] * f)[..., None, :]
    c, s = ang.cos() * mag, ang.sin() * mag
    y = x.clone()
    ia = slice(0, n // 2) if pairs == "half" else slice(0, n, 2)
    ib = slice(n // 2, n) if pairs == "half" else slice(1, n, 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def slot_of(layout, p, window=0, sinks=0):
    """Slot of position p in a window cache."""
    if layout == "ring" or p >= sinks:
        return sinks + (p - sinks) % window
    return p


def attended(layout, t, window=0, sinks=0, start=0):
    """Positions the token at t attends, itself included, ascending."""
    if t < 0:
        return []
    if layout == "paged":
        ps = range(t + 1)
    else:
        ps = sorted(set(range(min(sinks, t + 1))) | set(range(max(0, t - window + 1), t + 1)))
    return [p for p in ps if p >= start]


def attend(q, k, v, dist, see, scale, cap=0.0, slopes=None):
    """q [T, H, D], k / v [L, KV, D] float64, dist / see [T, L]; a row that sees nothing gives 0."""
    T, H, D = q.shape
    G = H // k.shape[1]
    if not T or not k.shape[0]:
        return torch.zeros_like(q), q.new_zeros(H, T, k.shape[0])
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("thd,lhd->htl", q, k) * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    if slopes is not None:
        s = s - slopes.double()[:, None, None] * dist[None].double()
    s = s.masked_fill(~see[None], -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = e.sum(-1, keepdim=True)
    w = torch.where(z > 0, e / z.clamp(min=1e-300), torch.zeros_like(e))
    return torch.einsum("htl,lhd->thd", w, v), w
