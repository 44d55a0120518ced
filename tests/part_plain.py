"""Plain forms of the operators on caches read or kept in part, for the tests: whole numbers for bounds,
selection and eviction, float64 for attention over any set of positions of each kv head."""

from __future__ import annotations

import math

import torch


def ends(k):
    """k [rows, D] (fp32 values): codes (largest, smallest) [2, D] and the step, as fp32 arithmetic gives them.
    A quotient of two fp32 numbers taken in float64 and rounded to fp32 is the correctly rounded quotient."""
    hi, lo = k.double().max(0).values, k.double().min(0).values
    step = (torch.maximum(hi.abs().max(), lo.abs().max()) / 127.0).float().double()
    if not step > 0:
        return torch.zeros(2, k.shape[1], dtype=torch.int8, device=k.device), step.float()
    codes = torch.stack([torch.ceil((hi / step).float()).clamp(max=127), torch.floor((lo / step).float()).clamp(min=-127)])
    return codes.to(torch.int8), step.float()


def query_codes(q):
    """q [H, D] -> codes int64, steps fp32 [H]."""
    step = (q.double().abs().amax(-1) / 127.0).float()
    safe = torch.where(step > 0, step, 1.0).double()
    codes = torch.where(step[:, None] > 0, (q.double() / safe[:, None]).float().round().clamp(-127, 127), 0.0)
    return codes.long(), step


def select(codes, steps, q, candidates, nb, k, first, recent, G):
    """Lists [KV] of chosen logical blocks: codes int8 [blocks, KV, 2, D] and steps [blocks, KV] indexed by logical
    block, candidates ascending."""
    qc, qs = query_codes(q)
    out = []
    for h in range(codes.shape[1]):
        ranked = []
        for lb in candidates:
            if lb < first or lb >= nb - recent:
                ranked.append((-math.inf, lb))
                continue
            best = -math.inf
            for x in range(h * G, h * G + G):
                u = torch.maximum(qc[x] * codes[lb, h, 0].long(), qc[x] * codes[lb, h, 1].long()).sum()
                best = max(best, float(u.float() * (qs[x] * steps[lb, h])))
            ranked.append((-best, lb))
        out.append(sorted(lb for _, lb in sorted(ranked)[:k]))
    return out


def attend(q, k, v, scale):
    """q [G, D], k / v [L, D] float64 -> out [G, D], weights [G, L] (nothing to attend: zeros)."""
    if not k.shape[0]:
        return torch.zeros_like(q), q.new_zeros(q.shape[0], 0)
    w = torch.softmax(q @ k.T * scale, -1)
    return w @ v, w


def evict(weights, table, pos, bs, keep, first, recent, refcount, free_list, free_count, num_blocks):
    """In place on Python lists; returns the blocks given back, ascending."""
    back = []
    for b, t in enumerate(pos):
        nb = 0 if t < 0 else min(t // bs + 1, len(table[b]))
        live = [lb for lb in range(nb) if table[b][lb] >= 0]
        loose = [lb for lb in live if first <= lb < nb - recent]

        def key(lb):
            w = weights[b][lb]
            return (1, 0.0, lb) if w != w else (0, w, lb)

        for lb in sorted(loose, key=key)[:max(0, len(live) - keep)]:
            p = table[b][lb]
            table[b][lb] = -1
            weights[b][lb] = 0.0
            refcount[p] -= 1
            if refcount[p] == 0:
                back.append(p)
    back.sort()
    return free_list[:free_count] + back + free_list[free_count + len(back):], free_count + len(back), back
