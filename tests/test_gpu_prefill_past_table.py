"""Chunks whose positions lie past the end of the block table: KVC_DEV_BAD_POSITION, and the tokens attend
their own sequence's blocks and the chunk, never the table's next row.  The table passed is the head of a
larger tensor whose further entries name blocks of their own, so that an entry read past the end shows in the
output and not as a fault."""

import math

import pytest
import torch

from tests import plain_ops as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("dtype,D,bs", [("bf16", 64, 16), ("bf16", 128, 8), ("bf16", 128, 64), ("bf16", 256, 32),
                                        ("i8", 128, 16), ("bf16", 128, 24)])
def test_positions_past_the_block_table(kvc, dtype, D, bs, scored):
    if scored and bs == 24:
        pytest.skip("modified scores take blocks that pack 64 rows")
    H, KV, T, maxb = 4, 2, 20, 5
    full = maxb * bs
    # inside, up to the end, across the end, at it, a few blocks past it, and at the end of the range
    pos0 = [full - T - 5, full - T, full - 7, full, full + 4 * bs + 3, 2 ** 31 - 1 - T]
    if bs == 24:
        pos0[5] = full + 300 * bs             # (that kernel walks every tile up to the position)
    B, pad = len(pos0), 64
    n_own = B * maxb
    blocks = n_own + 4
    d = kvc.make_desc("paged", "none", dtype, layers=1, batch=B, q_heads=H, kv_heads=KV, head_dim=D, block_size=bs,
                      num_blocks=blocks, max_blocks_per_seq=maxb)
    perm = torch.randperm(n_own, generator=torch.Generator().manual_seed(bs))
    whole = torch.full((B + pad, maxb), n_own, dtype=torch.int32)
    whole[:B] = perm.view(B, maxb).to(torch.int32)
    table = whole.cuda()[:B]
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = kvc.alloc_cache(d)
    if dtype == "i8":
        codes, scales = kvc.int8_views(d, cache)
        codes.copy_(torch.randint(-127, 128, codes.shape, generator=g, device="cuda").to(torch.int8))
        scales.fill_(1 / 64)
        rows = (codes[0].double() * scales[0].double()[..., None]).to(torch.bfloat16).double()
        scales[0, :, n_own:] = 100.0
    else:
        cache.copy_(torch.randn(cache.shape, generator=g, device="cuda"))
        rows = cache[0].double()
        cache[0, :, n_own:] = 100.0
    q, k, v = (torch.randn(B, T, n, D, generator=g, device="cuda").to(torch.bfloat16) for n in (H, KV, KV))
    pos = torch.tensor(pos0, dtype=torch.int32, device="cuda")
    ws = kvc.alloc_prefill_workspace(d, T)
    if scored:
        out = kvc.prefill_scored(d, cache, 0, q, k, v, pos, ws, kvc.make_score(), block_table=table)
    else:
        out = kvc.prefill(d, cache, 0, q, k, v, pos, ws, block_table=table)
    assert kvc.get_error(ws) == kvc.KVC_DEV_BAD_POSITION
    if dtype == "i8":
        x = []
        for y in (k, v):
            s = y.double().abs().amax(-1, keepdim=True).float() / 127
            x.append(((y.float() / s).round().clamp(-127, 127).double() * s.double()).to(torch.bfloat16).double())
        k64, v64 = x
    else:
        k64, v64 = k.double(), v.double()
    for b, n in enumerate(pos0):
        m = min(n, full)
        K, V = (rows[w][table[b].long()].permute(0, 2, 1, 3).reshape(full, KV, D)[:m] for w in range(2))
        t = torch.arange(n, n + T, device="cuda")
        own = torch.ones(T, dtype=torch.bool, device="cuda")
        if bs == 24:
            own = t < full                    # that kernel knows no chunk keys past the table either
        K, V = torch.cat([K, k64[b][own]]), torch.cat([V, v64[b][own]])
        p = torch.cat([torch.arange(m, device="cuda"), t[own]])
        want, w = plain.attend(q[b].double(), K, V, t[:, None] - p[None], p[None] <= t[:, None], D ** -0.5)
        weight = torch.einsum("htl,lhd->thd", w, V.abs().repeat_interleave(H // KV, 1))
        # scores: a query scaled and rounded to bf16 (2^-8 sum |q_i k_i| scale, twice in a weight); weights
        # as in the prefill tests (fp16 argument and result, bf16), the output half a step
        qk = float(torch.einsum("thd,lhd->htl", q[b].double().abs(), K.abs().repeat_interleave(H // KV, 1)).amax())
        rel = math.expm1(2 * 2.0 ** -8 * qk * D ** -0.5) + 2.0 ** -8 + 1.3e-2
        tol = rel * weight + 2.0 ** -8 * (want.abs() + rel * weight) + 1e-6
        assert ((out[b].double() - want).abs() <= tol).all(), (b, n)
