"""One paged sequence with num_splits set, above the number of decode CTAs too: every row is attended, by the
plain call, the step and the scored call.

Tolerance of the plain calls, relative to sum w |v|: weights rounded to bf16 (fp16 on INT8 caches) 2^-8,
fp32 statistics 1e-3, and the query rounded to bf16 after its scale: 2^-8 sum |q_i k_i| scale in a score,
twice that in a weight; the output half a step."""

import math

import pytest
import torch

from tests import plain_ops as plain
from tests import test_gpu_scored as scored
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


@pytest.mark.parametrize("num_splits", [0, 1, 9, 17, 64, 400, 5000])
@pytest.mark.parametrize("H,KV", [(40, 8), (8, 8), (4, 1)])
@pytest.mark.parametrize("dtype,D,n,bs", [("bf16", 64, 56, 20), ("bf16", 128, 700, 16), ("bf16", 256, 333, 64),
                                          ("i8", 128, 700, 16), ("f32", 64, 500, 16)])
def test_splits_of_one_sequence(kvc, dtype, D, n, bs, H, KV, num_splits):
    scored._decode(kvc, "paged", dtype, lens=(n,), H=H, KV=KV, D=D, bs=bs, num_splits=num_splits, cap=9.0, bias=True)
    c = Built(kvc, "paged", dtype, (n,), H, KV, D, bs=bs, num_splits=num_splits, qstd=1.0)
    k, v = c.rows(0, range(n))
    see = torch.ones(1, n, dtype=torch.bool, device="cuda")
    q = c.q[0].double()
    want, w = plain.attend(q[None], k, v, see, see, c.scale)
    weight = torch.einsum("htl,lhd->thd", w, v.abs().repeat_interleave(H // KV, 1))
    qk = float(torch.einsum("hd,lhd->hl", q.abs(), k.abs().repeat_interleave(H // KV, 1)).amax()) * c.scale
    rel = scored.REL[dtype] + (0.0 if dtype == "f32" else math.expm1(2 * 2.0 ** -8 * qk))
    for _ in range(2):
        out = kvc.decode_attention(c.d, c.cache, c.layer, c.q, c.pos, c.ws, block_table=c.table)
        scored._within(out[0], want[0], weight[0], rel, c.act)
    # the step appends its own token: the last row's values again (INT8: what the row holds, quantised anew)
    if dtype != "i8":
        row = [x[n - 1][None].to(c.act) for x in (k, v)]
        out = kvc.decode_step(c.d, c.cache, c.layer, c.q, row[0], row[1], c.pos, c.ws, block_table=c.table)
        scored._within(out[0], want[0], weight[0], rel, c.act)
    assert kvc.get_error(c.ws) == 0
