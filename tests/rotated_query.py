"""Decode attention of one query of each head whose rotation is done by the call, in float64, for the tests of the decode
calls on parts of a cache.

On a bf16 cache the rotated query enters the products rounded to bf16, here too, so that only values at a tie are allowed
for (draft_plain.rotated); on an INT8 cache it is rounded to fp16: a score is off by 2^-11 sum |q_i k_i| scale, which
enters a weight twice."""

from __future__ import annotations

import torch

from tests import draft_plain as draft
from tests import part_plain as part
from tests import plain_ops as plain


def attend(q, t, k, v, scale, dtype):
    """q [G, D] at position t, k / v [L, D] (float64) -> out, how far it may be off, weights [G, L], and how far a weight may
    be off relative to itself for the query's rounding [G, 1]."""
    if dtype == "bf16":
        qt, eq = (x[0] for x in draft.rotated(q[None], torch.tensor([t], device=q.device)))
        off = (eq @ k.abs().T).amax(-1, keepdim=True) * scale
    else:
        qt = plain.rotate(q[None], torch.tensor([t], device=q.device), plain.frequencies(q.shape[-1])[0], 1.0, "half")[0]
        off = (qt.abs() @ k.abs().T).amax(-1, keepdim=True) * scale * 2.0 ** -11
    out, w = part.attend(qt, k, v, scale)
    near = torch.expm1(2 * off)
    rel = draft.REL + near
    mass = w @ v.abs()
    return out, rel * mass + 2.0 ** -8 * (out.abs() + rel * mass) + 1e-6, w, near
