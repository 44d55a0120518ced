"""Scored prefill and shared-prefix decode within the bounds of their arithmetic, which takes fp32
exponentials.

For an output sum w_i v_i, relative to sum w_i |v_i|: each weight is rounded to bf16 before it meets v,
half a step, 2^-8; it comes from a score off by at most 2^-24 D sum |q_i k_i| scale (under 28 for these
inputs: 4.3e-4 at D = 256), which counts in numerator and denominator, and the rest is below 1e-4: the
exponential's 2^-22, its argument's rounding (2^-24 of under 40), a capped score's 6 2^-23 cap, the fp32 sums of
under 2000 keys, 16 at a time.  2^-8 + 1e-3 together, and the output's half step.  A baked query rounded to
bf16 after its rotation moves scores by 2^-8 sum |q_i k_i| scale more."""

import math

import pytest
import torch

from tests import plain_ops as plain
from tests import test_gpu_scored as scored
from tests import test_gpu_shared as shared
from tests.cache_builder import Built

pytestmark = pytest.mark.gpu

REL = 2.0 ** -8 + 1e-3
MORE = 1e-3 - 1.3e-2          # from the bound that the scored prefill's tests allow to REL


LAYOUTS = [("paged", dict(lens=(0, 50, 1333), bs=16)), ("ring", dict(lens=(0, 150, 2000), window=700)),
           ("sink_ring", dict(lens=(2, 150, 2000), window=700, sinks=4))]


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


@pytest.mark.parametrize("mods", scored.MODS + [dict(cap=40.0), dict(cap=200.0)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("layout,kw", LAYOUTS)
def test_prefill(kvc, mods, D, layout, kw):
    scored._prefill(kvc, layout, "bf16", T=97, D=D, more=MORE, **kw, **mods)


@pytest.mark.parametrize("mods", scored.MODS + [dict(cap=40.0), dict(cap=200.0)])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("layout,kw", LAYOUTS)
def test_prefill_int8(kvc, mods, D, layout, kw):
    """Rows as the kernel reads them: code * scale in fp32, then bf16 (one rounding of the exact product, as the
    scored prefill's own tests take it, sits a step apart next to a tie)."""
    H, KV, T = 8, 2, 97
    c = Built(kvc, layout, "i8", H=H, KV=KV, D=D, new=T, **kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    B = len(c.lens)
    q = (torch.randn(B, T, H, D, generator=g, device="cuda") * 2).to(torch.bfloat16)
    k, v = (torch.randn(B, T, KV, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos0 = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    slopes = scored._slopes(H) if mods.get("bias") else None
    cap = mods.get("cap", 0.0)
    ws = kvc.alloc_prefill_workspace(c.d, T)
    before, chunk = c.cache.clone(), torch.empty_like(c.cache)
    out = kvc.prefill_scored(c.d, c.cache, c.layer, q, k, v, pos0, ws, kvc.make_score(cap, slopes), block_table=c.table)
    # the chunk's codes and scales, from an append of it
    chunk.copy_(before)
    kvc.append(c.d, chunk, c.layer, k, v, pos0, ws, block_table=c.table)
    assert kvc.get_error(ws) == 0

    def rows(cache, b, ps):
        codes, scales = kvc.int8_views(c.d, cache)
        p = torch.as_tensor(ps, dtype=torch.long)
        if layout == "paged":
            i, r = c.table[b].cpu().long()[p // c.bs], p % c.bs
        else:
            i = torch.full_like(p, b)
            r = torch.tensor([plain.slot_of(layout, int(x), c.window, c.sinks) for x in p], dtype=torch.long)
        return [(codes[c.layer, w][i, :, r].float() * scales[c.layer, w][i, :, r][..., None]).to(torch.bfloat16).double()
                for w in range(2)]

    for b, n in enumerate(c.lens):
        old = plain.attended(layout, n - 1, c.window, c.sinks)
        new = list(range(n, n + T))
        K, V = (torch.cat([x, y]) for x, y in zip(rows(before, b, old), rows(chunk, b, new)))
        t = torch.arange(n, n + T, device="cuda")
        p = torch.cat([torch.tensor(old, dtype=torch.long, device="cuda"), t])
        see = p[None] <= t[:, None]
        if layout != "paged":
            see &= (p[None] < c.sinks) | (p[None] > t[:, None] - c.window)
        want, w = plain.attend(q[b].double(), K, V, t[:, None] - p[None], see, c.scale, cap, slopes)
        weight = torch.einsum("htl,lhd->thd", w, V.abs().repeat_interleave(H // KV, 1))
        scored._within(out[b], want, weight, REL, c.act)


@pytest.mark.parametrize("mods", [dict(cap=15.0), dict(bias=True), dict(cap=15.0, bias=True)])
@pytest.mark.parametrize("H,KV", [(8, 1), (6, 1), (10, 2), (8, 8)])
def test_prefill_documents_and_groups(kvc, mods, H, KV):
    docs = lambda b, i, n: max(n, 0) + (i // 90) * 90 if i >= 20 else n // 2
    scored._prefill(kvc, "paged", "bf16", lens=(0, 77, 300), T=300, H=H, KV=KV, docs=docs, more=MORE, **mods)
    scored._prefill(kvc, "ring", "bf16", lens=(0, 77, 900), T=300, H=H, KV=KV, docs=docs, window=400, more=MORE, **mods)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [8, 16, 64, 128])
def test_shared(kvc, D, bs):
    lens = [400, 290, 333, 257, 310, 41, 275]
    c, _, _, out = shared._run(kvc, lens, [0, 0, 1, 1, 1, -1, 1], [((0, 1), 256 // bs), ((2, 3, 4, 6), 256 // bs)], D=D,
                               bs=bs)
    shared._check(c, out, rel=REL)


@pytest.mark.parametrize("n,H,KV", [(2, 8, 2), (9, 8, 1), (33, 8, 1), (70, 8, 1), (130, 1, 1), (3, 128, 1), (9, 10, 2)])
def test_shared_columns(kvc, n, H, KV):
    c, _, _, out = shared._run(kvc, [1100 + 7 * (i % 40) for i in range(n)], [0] * n, [(range(n), 66)], H=H, KV=KV)
    shared._check(c, out, rel=REL)


def test_shared_baked(kvc):
    lens = [150, 131, 200]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 64, tables=shared._tables(lens, [((0, 1, 2), 8)], 16), rope="baked",
              qstd=1.0)
    c.baked = True
    ws = kvc.alloc_shared_workspace(c.d)
    out = kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, torch.zeros(3, dtype=torch.int32, device="cuda"),
                                      ws, c.table)
    qk = max(float(torch.einsum("hd,lhd->hl", c.q[b].double().abs() * 2 ** 0.5,
                                c.rows(b, range(n))[0].abs().repeat_interleave(4, 1)).amax())
             for b, n in enumerate(lens)) * c.scale
    shared._check(c, out, rel=REL + math.expm1(2 * 2.0 ** -8 * qk))
