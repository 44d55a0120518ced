"""kvc_tree_attention where a share of the work holds several segments of unequal length, one tile among them, at every
head dimension and with rotated keys.  A column of one tile (an idle or empty sequence) brings the second issuing warp of
a one-Q-tile draft no product: it has to skip that segment's q and find the next one's."""

import pytest
import torch

from tests import draft_plain as draft
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


class Batch:
    def __init__(self, kvc, layout, lens, T, H, KV, D, rope, padded=True, seed=0, **kw):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kvc, self.T, self.rope = kvc, T, rope
        self.c = c = Built(kvc, layout, "bf16", lens, H, KV, D, rope=rope, layers=1, **kw)
        B = len(lens)
        self.parents = [draft.random_tree(T, b, padded and b % 3 == 1) for b in range(B)]
        self.parent = torch.tensor(self.parents, dtype=torch.int32, device="cuda")
        self.q = (torch.randn(B, T, H, D, generator=g, device="cuda") * 0.75).to(torch.bfloat16)
        self.k, self.v = (torch.randn(B, T, KV, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        self.pos0 = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.ws = kvc.alloc_tree_workspace(c.d, T)

    def run(self, out=None):
        c = self.c
        if out is None:
            out = torch.full_like(self.q, float("nan"))
        return self.kvc.tree_attention(c.d, c.cache, c.layer, self.q, self.k, self.v, self.pos0, self.parent, self.ws, c.table,
                                       out=out)

    def check(self, out):
        c = self.c
        for b, n in enumerate(c.lens):
            ps = sorted(c.kv[b])
            kc, vc = c.rows(b, ps) if ps else (self.q.new_zeros(0, c.KV, c.D, dtype=torch.float64),) * 2
            tok, want, tol = draft.attend(self.q[b].double(), self.k[b].double(), self.v[b].double(), self.parents[b], n, ps, kc,
                                          vc, c.layout, c.window, c.sinks, c.scale, self.rope)
            draft.compare(out[b], self.T, tok, want, tol, b)

    def repeat(self, first, times):
        out = torch.empty_like(first)
        same = torch.ones((), dtype=torch.bool, device="cuda")
        for _ in range(times):
            self.run(out)
            same &= (out.view(torch.int16) == first.view(torch.int16)).all()
        assert bool(same) and self.kvc.get_error(self.ws) == 0


# 150 sequences x 2 kv heads, 31 tiles for every six sequences: ten tiles and more in a share, two to four segments
LENS = [500, 0, 300, -1, 64, 700] * 25


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rope", ["none", "baked"])
def test_unequal_segments(kvc, D, rope):
    s = Batch(kvc, "paged", LENS, 6, 8, 2, D, rope)
    out = s.run()
    assert kvc.get_error(s.ws) == 0
    s.check(out)
    s.repeat(out, 300)


@pytest.mark.parametrize("rope", ["none", "baked"])
@pytest.mark.parametrize("lens", [[0, 400] * 60, [-1, 0, 0, 1000] * 40, [64 * (i % 4) for i in range(200)],
                                  [0] * 300 + [3000] * 8, [70, 0, 0, 0, 130] * 40], ids=lambda x: f"{x[:5]}x{len(x)}")
def test_segments_of_one_tile(kvc, lens, rope):
    """One Q tile at head_dim 128: runs of one-tile columns, alone, before and behind longer ones."""
    s = Batch(kvc, "paged", lens, 4, 4, 2, 128, rope)
    out = s.run()
    assert kvc.get_error(s.ws) == 0
    s.check(out)
    s.repeat(out, 300)


@pytest.mark.parametrize("rope", ["none", "baked"])
def test_unequal_rings(kvc, rope):
    """Rings that are idle, empty, part full and wrapped."""
    s = Batch(kvc, "ring", [-1, 0, 10, 300, 1000, 70, 512, 0] * 18, 8, 16, 4, 128, rope, window=512)
    out = s.run()
    assert kvc.get_error(s.ws) == 0
    s.check(out)
    s.repeat(out, 300)
