"""Chunked prefill far into a sequence: the query's rotation keeps its angle at any position that an
int32 holds, in kvc_prefill (baked and read-time RoPE) and kvc_prefill_scored (baked).

Queries are zero outside their first eight rotation pairs, whose frequencies are the highest.

Tolerance, for an output sum w_i v_i: a query is rounded to bf16 after its rotation and, in plain
prefill, its scale, and with read-time RoPE a key after its own (half a step, 2^-8): scores are off by
2^-8 sum |q_i k_i| scale each, of the rotated values, and a weight by twice that.  A plain weight's base-2 argument is rounded to fp16, 2^-7 below 32, in numerator
and denominator: 2 ln 2 2^-8 each, and the result 2^-11 twice; bf16 weights 2^-8, fp32 statistics
1e-3, the output half a step."""

import math

import pytest
import torch

from tests import plain_ops as plain
from tests.cache_builder import Built

pytestmark = pytest.mark.gpu

PAIRS = 8
FAR = (1 << 20, (1 << 24) + 12345, 1 << 30, 2 ** 31 - 1 - 40)


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _few_pairs(x):
    D = x.shape[-1]
    keep = torch.zeros(D, dtype=torch.bool, device=x.device)
    keep[:PAIRS] = keep[D // 2:D // 2 + PAIRS] = True
    return torch.where(keep, x, torch.zeros_like(x))


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("rope", ["baked", "read_time"])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("i8", 128), ("i8", 256)])
def test_prefill_rotates_queries_exactly(kvc, dtype, D, rope, scored):
    if scored and rope == "read_time":
        pytest.skip("modified scores take no read-time RoPE")
    H, KV, T, S, W = 4, 2, 40, 4, 92
    B = len(FAR)
    c = Built(kvc, "sink_ring", dtype, FAR, H, KV, D, window=W, sinks=S, rope=rope)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = _few_pairs(torch.randn(B, T, H, D, generator=g, device="cuda") * math.sqrt(D) / 4).to(torch.bfloat16)
    k, v = (torch.randn(B, T, KV, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos0 = torch.tensor(FAR, dtype=torch.int32, device="cuda")
    ws = kvc.alloc_prefill_workspace(c.d, T)
    after = c.cache.clone()
    kvc.append(c.d, after, c.layer, k, v, pos0, ws)
    if scored:
        out = kvc.prefill_scored(c.d, c.cache, c.layer, q, k, v, pos0, ws, kvc.make_score())
    else:
        out = kvc.prefill(c.d, c.cache, c.layer, q, k, v, pos0, ws)
    assert kvc.get_error(ws) == 0
    # the chunk's rows as the cache holds them
    slots = torch.tensor([[plain.slot_of("sink_ring", p + i, W, S) for i in range(T)] for p in FAR], device="cuda")
    if dtype == "i8":
        codes, scales = kvc.int8_views(c.d, after)
        stored = [torch.stack([(codes[c.layer, w][b, :, slots[b]].double() *
                                scales[c.layer, w][b, :, slots[b]].double()[..., None]).transpose(0, 1)
                               for b in range(B)]) for w in range(2)]
    else:
        stored = [torch.stack([after[c.layer, w][b, :, slots[b]].double().transpose(0, 1) for b in range(B)])
                  for w in range(2)]
    freq, _ = plain.frequencies(D)
    for b, n in enumerate(FAR):
        old = plain.attended("sink_ring", n - 1, W, S)
        kc, vc = c.rows(b, old)
        K, V = torch.cat([kc, stored[0][b]]), torch.cat([vc, stored[1][b]])
        if dtype == "i8":          # as the kernel reads them: bf16 of code * scale
            K, V = K.to(torch.bfloat16).double(), V.to(torch.bfloat16).double()
        t = torch.arange(n, n + T, device="cuda")
        p = torch.cat([torch.tensor(old, device="cuda"), t])
        see = (p[None] <= t[:, None]) & ((p[None] < S) | (p[None] > t[:, None] - W))
        x = q[b].double()
        rot = lambda y, at: plain.rotate(y, at, freq, 1.0, "half")
        qt = rot(x, t)
        qk = lambda y, z: torch.einsum("thd,lhd->htl", y, z.repeat_interleave(H // KV, 1))
        if rope == "read_time":    # sink keys at their index, with the query at its own there
            K = rot(K, p)
            s, mag = qk(qt, K), qk(qt.abs(), K.abs())
            qs = rot(x, torch.full_like(t, S + W - 1))
            s[..., :S], mag[..., :S] = qk(qs, K[:S]), qk(qs.abs(), K[:S].abs())
        else:
            s, mag = qk(qt, K), qk(qt.abs(), K.abs())
        w = torch.softmax((s * c.scale).masked_fill(~see[None], -math.inf), -1)
        want = torch.einsum("htl,lhd->thd", w, V.repeat_interleave(H // KV, 1))
        weight = torch.einsum("htl,lhd->thd", w, V.abs().repeat_interleave(H // KV, 1))
        rounds = 2 if rope == "read_time" else 1
        rel = math.expm1(2 * rounds * 2.0 ** -8 * float(mag.masked_fill(~see[None], 0).amax()) * c.scale)
        rel += 2.0 ** -8 + 1e-3
        if not scored:
            rel += 2 * math.log(2) * 2.0 ** -7 + 2.0 ** -10
        tol = rel * weight + 2.0 ** -8 * (want.abs() + rel * weight) + 1e-6
        err = (out[b].double() - want).abs()
        assert torch.isfinite(out[b].float()).all()
        assert (err <= tol).all(), (n, float((err / tol).max()))
