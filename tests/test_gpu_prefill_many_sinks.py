"""Chunked prefill with read-time RoPE over more attention sinks than a tile of keys holds (64): every sink is
attended, at its index in the compacted cache, with the query at its own.

Tolerance as in the tests of far positions: queries (after rotation and scale) and keys (after rotation) are
rounded to bf16, a weight's base-2 argument to fp16 (2^-7 below 32) and the result, the weight to bf16."""

import math

import pytest
import torch

from tests import plain_ops as plain
from tests.cache_builder import Built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


@pytest.mark.parametrize("S,W", [(64, 64), (68, 60), (132, 60), (200, 100)])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("i8", 128), ("i8", 256)])
def test_many_sinks(kvc, dtype, D, S, W):
    H, KV, T = 4, 2, 40
    lens = (0, 30, 66, 131, S, S + W - 10, S + W + 500)
    B = len(lens)
    c = Built(kvc, "sink_ring", dtype, lens, H, KV, D, window=W, sinks=S, rope="read_time")
    g = torch.Generator(device="cuda").manual_seed(1)
    q = (torch.randn(B, T, H, D, generator=g, device="cuda") * 0.7).to(torch.bfloat16)
    k, v = (torch.randn(B, T, KV, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos0 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = kvc.alloc_prefill_workspace(c.d, T)
    out = kvc.prefill(c.d, c.cache, c.layer, q, k, v, pos0, ws)
    assert kvc.get_error(ws) == 0
    k64, v64 = k.double(), v.double()
    if dtype == "i8":
        x = []
        for y in (k, v):
            s = y.double().abs().amax(-1, keepdim=True).float() / 127
            x.append(((y.float() / s).round().clamp(-127, 127) * s).to(torch.bfloat16).double())
        k64, v64 = x
    freq, _ = plain.frequencies(D)
    rot = lambda y, at: plain.rotate(y, at, freq, 1.0, "half")
    qk = lambda y, z: torch.einsum("thd,lhd->htl", y, z.repeat_interleave(H // KV, 1))
    for b, n in enumerate(lens):
        old = plain.attended("sink_ring", n - 1, W, S)
        kc, vc = c.rows(b, old) if old else (k64[b, :0], v64[b, :0])
        if dtype == "i8" and old:
            kc, vc = kc.to(torch.bfloat16).double(), vc.to(torch.bfloat16).double()
        K, V = torch.cat([kc, k64[b]]), torch.cat([vc, v64[b]])
        t = torch.arange(n, n + T, device="cuda")
        p = torch.cat([torch.tensor(old, dtype=torch.long, device="cuda"), t])
        see = (p[None] <= t[:, None]) & ((p[None] < S) | (p[None] > t[:, None] - W))
        Kr, x = rot(K, p), q[b].double()
        qt, qs = rot(x, t), rot(x, t.clamp(max=S + W - 1))
        sink = (p < S)[None, None]
        s = torch.where(sink, qk(qs, Kr), qk(qt, Kr)) * c.scale
        mag = torch.maximum(qk(qs.abs(), Kr.abs()), qk(qt.abs(), Kr.abs())) * c.scale
        w = torch.softmax(s.masked_fill(~see[None], -math.inf), -1)
        want = torch.einsum("htl,lhd->thd", w, V.repeat_interleave(H // KV, 1))
        weight = torch.einsum("htl,lhd->thd", w, V.abs().repeat_interleave(H // KV, 1))
        rel = math.expm1(2 * 2 * 2.0 ** -8 * float(mag.masked_fill(~see[None], 0).amax()))
        rel += 2.0 ** -8 + 1e-3 + 2 * math.log(2) * 2.0 ** -7 + 2.0 ** -10
        if dtype == "i8":          # a value next to a tie of its two roundings sits a step away
            rel += 2.0 ** -7
        tol = rel * weight + 2.0 ** -8 * (want.abs() + rel * weight) + 1e-6
        err = (out[b].double() - want).abs()
        assert torch.isfinite(out[b].float()).all()
        assert (err <= tol).all(), (n, float((err / tol).max()))
