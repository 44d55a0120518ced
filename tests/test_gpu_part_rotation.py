"""Decode over selected blocks and with block weights on caches of rotated keys: the query at its own position, against
float64 that rounds it as the kernel does (test_rotated_query_cpu.py shows that any other position is seen)."""

import pytest
import torch

from tests import rotated_query as rotated
from tests.cache_builder import Built

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 64, 3, 1, 8), ("bf16", 128, 8, 2, 16), ("bf16", 256, 6, 2, 20), ("i8", 128, 8, 4, 16), ("i8", 256, 6, 2, 8)]


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


@pytest.mark.parametrize("dtype,D,H,KV,bs", SHAPES)
def test_selected(kvc, dtype, D, H, KV, bs):
    lens = [1, 5 * bs, 30 * bs - 1, 17 * bs + 3]
    c = Built(kvc, "paged", dtype, lens, H, KV, D, bs=bs, rope="baked", qstd=1.0)
    g = torch.Generator().manual_seed(D)
    lists = [[sorted(torch.randperm(-(-n // bs), generator=g)[:6].tolist()) for _ in range(KV)] for n in lens]
    blocks = torch.tensor([[x + [-1] * (6 - len(x)) for x in row] for row in lists], dtype=torch.int32, device="cuda")
    ws = kvc.alloc_select_workspace(c.d, 6)
    out = kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, blocks, ws, c.table)
    G = H // KV
    for b, n in enumerate(lens):
        for h in range(KV):
            k, v = c.rows(b, [p for lb in lists[b][h] for p in range(lb * bs, min(n, lb * bs + bs))])
            want, tol, _, _ = rotated.attend(c.q[b, h * G:h * G + G].double(), n - 1, k[:, h], v[:, h], c.scale, dtype)
            err = (out[b, h * G:h * G + G].double() - want).abs()
            assert (err <= tol).all(), (b, h, float((err / tol).max()))
    assert kvc.get_error(ws) == 0


@pytest.mark.parametrize("dtype,D,H,KV,bs", SHAPES)
@pytest.mark.parametrize("batch", [1, 4])
def test_weighed(kvc, dtype, D, H, KV, bs, batch):
    """(one sequence plans for itself, a batch has a planning kernel)"""
    lens = [30 * bs - 1, 1, 5 * bs, 17 * bs + 3][:batch]
    c = Built(kvc, "paged", dtype, lens, H, KV, D, bs=bs, rope="baked", qstd=1.0)
    ws = kvc.alloc_weighed_workspace(c.d)
    weights = torch.zeros(c.table.shape, device="cuda")
    out = kvc.decode_attention_weighed(c.d, c.cache, c.layer, c.q, c.pos, weights, ws, c.table, decay=0.0)
    G = H // KV
    for b, n in enumerate(lens):
        add, allow = (torch.zeros(c.table.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
        lb = torch.arange(n, device="cuda") // bs
        k, v = c.rows(b, range(n))
        for h in range(KV):
            want, tol, w, near = rotated.attend(c.q[b, h * G:h * G + G].double(), n - 1, k[:, h], v[:, h], c.scale, dtype)
            err = (out[b, h * G:h * G + G].double() - want).abs()
            assert (err <= tol).all(), (b, h, float((err / tol).max()))
            add.index_add_(0, lb, w.sum(0))
            allow.index_add_(0, lb, (w * near).sum(0))
        # besides the query: fp32 scores of D products (|q k| scale below 40 here), exponentials, sums over heads and rows
        allow += add * (2 * D * 2.0 ** -24 * 40 + (H + bs + 64) * 2.0 ** -24 + 2.0 ** -20) + 1e-7
        err = (weights[b].double() - add).abs()
        assert (err <= allow).all(), (b, float((err / allow).max()))
    assert kvc.get_error(ws) == 0
