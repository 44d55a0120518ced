"""A tree of drafted tokens in float64, with its rotated rows rounded as they are stored, for the tests of
kvc_tree_attention.

A weight enters the second product rounded to bf16 (2^-8 of it), fp32 scores and statistics leave 1e-3 of
sum w |v| at most, and the output is rounded to bf16 once.  With baked RoPE q and the draft's keys are rounded to bf16
after their rotation, here too: what is left of that is the fp32 rotation's own error, which can bring a value to the
other side of a tie.  An angle is off by 2e-7 at most, its sine and cosine by as much again, products and their sum by
three halves of 2^-23: 6e-7 (|x1| + |x2|) for a value made of x1 and x2.  Only values that close to a tie can differ,
by the step between their two candidates; the score's error from them enters a weight twice."""

from __future__ import annotations

import math

import torch

from tests import plain_ops as plain

REL = 2.0 ** -8 + 1e-3


def lines(parent):
    """The tokens each token attends in the draft, root first (None: no token)."""
    out = []
    for i, p in enumerate(parent):
        if p == -1:
            out.append([i])
        elif 0 <= p < i and out[p] is not None:
            out.append(out[p] + [i])
        else:
            out.append(None)
    return out


def rotated(x, pos):
    """x [n, heads, D] (bf16 values, float64) at positions pos [n] -> the stored values, and how far each may be off."""
    D = x.shape[-1]
    y = plain.rotate(x, pos, plain.frequencies(D)[0], 1.0, "half")
    size = x.abs()
    off = 6e-7 * (size + size.roll(D // 2, -1))
    kept, low, high = (z.to(torch.bfloat16).double() for z in (y, y - off, y + off))
    return kept, high - low


def attend(q, k, v, parent, n, ps, kc, vc, layout, window, sinks, scale, rope, plant=""):
    """One sequence: q [T, H, D], k / v [T, KV, D] of the draft (float64), n tokens in the cache of which positions ps
    (ascending) hold rows kc / vc [len(ps), KV, D].  Returns the tokens that there are, their outputs and how far each
    value may be off.  `plant`: a mistake in the rotation, for a test of the tolerances."""
    tok = [i for i, line in enumerate(lines(parent)) if line is not None]
    way = lines(parent)
    dev = q.device
    if not tok or n < 0:
        return [], None, None
    depth = torch.tensor([len(way[i]) - 1 for i in tok], device=dev)
    at = {t: j for j, t in enumerate(tok)}
    see = torch.zeros(len(tok), len(ps) + len(tok), dtype=torch.bool, device=dev)
    for j, i in enumerate(tok):
        there = set(plain.attended(layout, n + len(way[i]) - 1, window, sinks))
        see[j, :len(ps)] = torch.tensor([p in there for p in ps], dtype=torch.bool, device=dev)
        see[j, [len(ps) + at[a] for a in way[i]]] = True
    qt, kt, vt = q[tok], k[tok], v[tok]
    eq, ek = torch.zeros_like(qt), torch.zeros_like(kt)
    if rope == "baked":
        qt, eq = rotated(qt, n + depth + (plant == "q one further"))
        if plant == "keys at pos0":
            depth = depth * 0
        if plant != "keys as they came":
            kt, ek = rotated(kt, n + depth)
    kk, vv, ee = torch.cat([kc, kt]), torch.cat([vc, vt]), torch.cat([torch.zeros_like(kc), ek])
    out, w = plain.attend(qt, kk, vv, see, see, scale)
    G = q.shape[1] // k.shape[1]
    wide = [x.abs().repeat_interleave(G, 1) for x in (kk, vv, ee)]
    mass = torch.einsum("htl,lhd->thd", w, wide[1])
    off = torch.einsum("thd,lhd->thl", eq, wide[0] + wide[2]) + torch.einsum("thd,lhd->thl", qt.abs(), wide[2])
    rel = REL + torch.expm1(2 * scale * off.masked_fill(~see[:, None], 0.0).amax(-1, keepdim=True))
    return tok, out, rel * mass + 2.0 ** -8 * (out.abs() + rel * mass) + 1e-6


def compare(got, T, tok, want, tol, where=""):
    """got [T, H, D]: within tol of want at the tokens, zeros elsewhere."""
    for i in range(T):
        if i not in tok:
            assert not got[i].any(), (where, i)
    if tok:
        err = (got[tok].double() - want).abs()
        assert torch.isfinite(got[tok]).all(), where
        assert (err <= tol).all(), (where, float((err / tol).max()))


def random_tree(T, seed, padded=False):
    g = torch.Generator().manual_seed(seed)
    p = [max(-1, i - 1 - int(torch.randint(0, 6, (1,), generator=g))) for i in range(T)]
    if padded:
        for i in range(T):
            if i % 5 == 3 or i >= T - T // 4:
                p[i] = -2 - i
    return p
