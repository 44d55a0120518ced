"""kvc_tree_attention on the GPU against the formula in float64, and a verification loop with kvc_append_path.

A weight enters the second product rounded to bf16 (2^-8 of it), fp32 scores and statistics leave 1e-3 of
sum w |v| at most, and the output is rounded to bf16 once.  With baked RoPE q and the draft's keys are rounded to
bf16 after their rotation: scores off by 2^-8 sum |q_i k_i| scale for each, twice in a weight."""

import math

import pytest
import torch

from tests import part_plain as part
from tests import plain_ops as plain
from tests.cache_builder import Built

pytestmark = pytest.mark.gpu

REL = 2.0 ** -8 + 1e-3


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _lines(parent):
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


def _tree(T, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "chain":
        return list(range(-1, T - 1))
    if kind == "star":
        return [-1] * T
    if kind == "binary":
        return [(i - 1) // 2 if i else -1 for i in range(T)]
    p = [max(-1, i - 1 - int(torch.randint(0, 6, (1,), generator=g))) for i in range(T)]
    if kind == "padded":
        for i in range(T):
            if i % 5 == 3 or i >= T - T // 4:
                p[i] = -2 - i
    return p


class Draft:
    """A cache of `lens` tokens a sequence and a draft of T tokens; padding tokens hold NaN."""

    def __init__(self, kvc, layout, lens, T, parents, H=8, KV=2, D=128, rope="none", **kw):
        g = torch.Generator(device="cuda").manual_seed(T)
        self.c = c = Built(kvc, layout, "bf16", lens, H, KV, D, rope=rope, **kw)
        B = len(lens)
        self.parents, self.T, self.rope = parents, T, rope
        self.q = (torch.randn(B, T, H, D, generator=g, device="cuda") * 1.5).to(torch.bfloat16)
        self.k, self.v = (torch.randn(B, T, KV, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        for b, par in enumerate(parents):
            for i, line in enumerate(_lines(par)):
                if line is None or lens[b] < 0:
                    for x in (self.q, self.k, self.v):
                        x[b, i] = float("nan")
        self.parent = torch.tensor(parents, dtype=torch.int32, device="cuda")
        self.pos0 = _i32(*lens)
        self.ws = kvc.alloc_tree_workspace(c.d, T)

    def run(self, kvc, valid=None, calls=2):
        c, first = self.c, None
        out = torch.empty_like(self.q)
        for _ in range(calls):
            out.fill_(float("nan"))
            kvc.tree_attention(c.d, c.cache, c.layer, self.q, self.k, self.v, self.pos0, self.parent, self.ws, c.table,
                               valid_bits=valid, out=out)
            # the same bits (NaN where a sequence past its table attends rows that hold no token)
            assert first is None or torch.equal(first.view(torch.int16), out.view(torch.int16))
            first = out.clone()
        return out

    def check(self, out, dead=(), skip=()):
        c = self.c
        G = c.H // c.KV
        freq = plain.frequencies(c.D)[0]
        kept = {}
        table = self.table if c.layout == "paged" else None
        for b, n in enumerate(c.lens):
            if b in skip:
                continue
            for i, line in enumerate(_lines(self.parents[b])):
                got = out[b, i].double()
                if line is None or n < 0:
                    assert not out[b, i].any(), (b, i)
                    continue
                t = n + len(line) - 1
                ps = [p for p in plain.attended(c.layout, t, c.window, c.sinks) if p < n]
                if c.layout == "paged":
                    ps = [p for p in ps if 0 <= table[b][p // c.bs] < c.d.num_blocks and table[b][p // c.bs] not in dead]
                kd, vd = self.k[b, line].double(), self.v[b, line].double()
                q = self.q[b, i].double()
                if self.rope == "baked":
                    kd = plain.rotate(kd, torch.arange(n, n + len(line), device="cuda"), freq, 1.0, "half")
                    q = plain.rotate(q, torch.tensor(t, device="cuda"), freq, 1.0, "half")
                if ps:
                    if (b, ps[0], len(ps)) not in kept:          # (positions of one sequence: whole runs but for sinks)
                        kept[b, ps[0], len(ps)] = (ps, c.rows(b, ps))
                    same, (k, v) = kept[b, ps[0], len(ps)]
                    if same != ps:
                        k, v = c.rows(b, ps)
                    kd, vd = torch.cat([k, kd]), torch.cat([v, vd])
                see = torch.ones(1, kd.shape[0], dtype=torch.bool, device="cuda")
                want, w = plain.attend(q[None], kd, vd, see, see, c.scale)
                mass = torch.einsum("htl,lhd->thd", w, vd.abs().repeat_interleave(G, 1))[0]
                rel = REL
                if self.rope == "baked":
                    qk = float(torch.einsum("hd,lhd->hl", q.abs(), kd.abs().repeat_interleave(G, 1)).max()) * c.scale
                    rel += math.expm1(4 * 2.0 ** -8 * qk)
                tol = rel * mass + 2.0 ** -8 * (want[0].abs() + rel * mass) + 1e-6
                err = (got - want[0]).abs()
                assert torch.isfinite(got).all(), (b, i)
                assert (err <= tol).all(), (b, i, float((err / tol).max()))

    @property
    def table(self):
        return self.c.table.tolist()


KINDS = ["chain", "star", "binary", "random", "padded"]


def _mixed(T, n):
    return [_tree(T, KINDS[b % 5], seed=b) for b in range(n)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 2, 5, 16, 31, 33, 64])
def test_paged(kvc, D, T):
    d = Draft(kvc, "paged", [130, 64, 1, 0, 300], T, _mixed(T, 5), D=D)
    d.check(d.run(kvc))
    assert kvc.get_error(d.ws) == 0


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 1), (10, 2), (16, 1), (14, 2), (4, 4), (128, 1), (40, 1)])
@pytest.mark.parametrize("T", [3, 20, 64])
def test_head_groups(kvc, H, KV, T):
    """Rows of one Q tile, of two, of several columns; groups that leave rows of a tile empty."""
    d = Draft(kvc, "paged", [150, 40], T, _mixed(T, 2), H=H, KV=KV, D=64)
    d.check(d.run(kvc))


def test_many_columns_of_head_dim_256(kvc):
    d = Draft(kvc, "paged", [150, 70], 64, _mixed(64, 2), H=12, KV=1, D=256)
    d.check(d.run(kvc))


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_blocks_and_absent_blocks(kvc, bs):
    lens = [400, 290, 333]
    d = Draft(kvc, "paged", lens, 9, _mixed(9, 3), bs=bs)
    t = d.table
    d.c.table[0, 1] = -1
    if lens[2] // bs > 6:
        d.c.table[2, 3:5] = -1
    dead = [t[1][0], t[1][290 // bs], t[0][2]]
    mask = torch.ones(d.c.d.num_blocks, dtype=torch.bool)
    mask[dead] = False
    d.check(d.run(kvc, kvc.pack_valid_bits(mask).cuda()), dead)
    d.check(d.run(kvc))
    d.c.table.fill_(-1)                       # nothing of the cache: the draft alone
    d.check(d.run(kvc))
    assert kvc.get_error(d.ws) == 0


@pytest.mark.parametrize("window,sinks", [(100, 0), (96, 4), (37, 70), (64, 0), (300, 1), (20, 3), (9, 0)])
@pytest.mark.parametrize("T", [1, 9, 20])
def test_windows(kvc, window, sinks, T):
    """Caches not yet full, just full, and wrapped at every place; deep tokens lose the oldest keys."""
    T = min(T, window)
    C = window + sinks
    lens = [0, 1, sinks, C - 1, C, C + 1, C + window // 2, 3 * C + 7, 5000]
    d = Draft(kvc, "sink_ring" if sinks else "ring", lens, T, _mixed(T, len(lens)), window=window, sinks=sinks, H=4, KV=2,
              D=64)
    d.check(d.run(kvc))
    assert kvc.get_error(d.ws) == 0


@pytest.mark.parametrize("D", [128, 256])
def test_windows_of_other_head_dims_and_chains(kvc, D):
    lens = [257, 200, 1000]
    d = Draft(kvc, "sink_ring", lens, 40, [_tree(40, "chain")] * 3, window=200, sinks=5, H=6, KV=2, D=D)
    d.check(d.run(kvc))


@pytest.mark.parametrize("T", [1, 8, 64])
def test_long_sequences(kvc, T):
    """One sequence cut into shares; a batch whose columns are cut too."""
    d = Draft(kvc, "paged", [20000], T, [_tree(T, "random")], H=4, KV=1, D=64, bs=64)
    d.check(d.run(kvc))
    d = Draft(kvc, "ring", [9000, 5000], T, [_tree(T, "binary"), _tree(T, "padded")], H=8, KV=8, D=64, window=4096)
    d.check(d.run(kvc))


def test_many_sequences(kvc):
    n = 200
    d = Draft(kvc, "paged", [(i * 37) % 150 for i in range(n)], 6, _mixed(6, n), H=4, KV=1, D=64, bs=8)
    d.check(d.run(kvc))


@pytest.mark.parametrize("layout", ["paged", "sink_ring"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_baked_rope(kvc, layout, D):
    lens = [150, 131, 260]
    kw = dict(window=100, sinks=4) if layout == "sink_ring" else {}
    d = Draft(kvc, layout, lens, 12, _mixed(12, 3), rope="baked", D=D, **kw)
    d.q.mul_(0.5)
    d.check(d.run(kvc))


def test_idle_bad_parents_and_positions(kvc):
    lens = [100, 60, 90, 40]
    bad = [[-1, 0, 2, 1, 9, 3], [0, -1, 1, 3, 2 ** 31 - 1, 2], [-1, 0, 1, 2, 3, 4], [-1, -2 ** 31, 1, 0, 0, 3]]
    d = Draft(kvc, "paged", lens, 6, bad)
    d.pos0 = _i32(100, 60, -1, 40)
    out = d.run(kvc)
    assert kvc.get_error(d.ws) == kvc.KVC_DEV_BAD_ENTRY
    assert not out[2].any()
    d.check(out, skip=(2,))
    d = Draft(kvc, "paged", lens, 6, _mixed(6, 4))
    d.pos0 = _i32(100, 60, 90, 10 ** 9)
    out = d.run(kvc)
    assert kvc.get_error(d.ws) == kvc.KVC_DEV_BAD_POSITION
    d.check(out, skip=(3,))
    d.c.table[1, 2] = d.c.d.num_blocks + 9
    d.pos0 = _i32(*lens)
    out = d.run(kvc)
    assert kvc.get_error(d.ws) == kvc.KVC_DEV_BAD_BLOCK
    d.check(out)


def test_a_nan_query_stays_in_its_rows(kvc):
    d = Draft(kvc, "paged", [300, 200], 10, _mixed(10, 2))
    ref = d.run(kvc)
    d.q[0, 4, 3, 7] = float("nan")
    out = d.run(kvc, calls=1)
    assert torch.isnan(out[0, 4, 3]).all()
    out[0, 4, 3] = ref[0, 4, 3]
    assert torch.equal(out, ref)


def test_a_chain_equals_prefill(kvc):
    """A draft without branches is a chunk: kvc_prefill's outputs, to the rounding of their sums."""
    T = 24
    d = Draft(kvc, "ring", [500, 90], T, [_tree(T, "chain")] * 2, window=128)
    out = d.run(kvc)
    pws = kvc.alloc_prefill_workspace(d.c.d, T)
    ref = kvc.prefill(d.c.d, d.c.cache, d.c.layer, d.q, d.k, d.v, d.pos0, pws)
    assert float((ref.float() - out.float()).abs().max()) < 6e-2


def test_workspace_serves_decode_calls(kvc):
    d = Draft(kvc, "paged", [300, 200], 10, _mixed(10, 2))
    ref = d.run(kvc)
    for _ in range(2):
        one = kvc.decode_attention(d.c.d, d.c.cache, d.c.layer, d.c.q, d.c.pos, d.ws, block_table=d.c.table)
        two = kvc.decode_attention(d.c.d, d.c.cache, d.c.layer, d.c.q, d.c.pos, d.c.ws, block_table=d.c.table)
        assert torch.equal(one, two) and torch.equal(d.run(kvc, calls=1), ref)


def test_offsets_past_32_bits(kvc):
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=2, q_heads=8, kv_heads=8, head_dim=128, block_size=16,
                      num_blocks=140000, max_blocks_per_seq=6)
    cache = kvc.alloc_cache(d)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = _i32(139999, 5, 70000, 139990, 1, 2, 139998, 7, 70001, 139990, 139991, 3).view(2, 6)
    for blk in table.flatten().unique().tolist():
        cache[0, :, blk] = torch.randn(2, 8, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = (torch.randn(2, 5, 8, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    par = [[-1, 0, 0, 1, -1], [-1, 0, 1, 2, 3]]
    ws = kvc.alloc_tree_workspace(d, 5)
    out = kvc.tree_attention(d, cache, 0, q, k, v, _i32(70, 95), torch.tensor(par, dtype=torch.int32, device="cuda"), ws, table)
    for b, n in enumerate((70, 95)):
        rows = cache[0, :, table[b].long()].double()
        kc, vc = (rows[i].permute(0, 2, 1, 3).reshape(96, 8, 128)[:n] for i in range(2))
        for i, line in enumerate(_lines(par[b])):
            kk, vv = torch.cat([kc, k[b, line].double()]), torch.cat([vc, v[b, line].double()])
            see = torch.ones(1, kk.shape[0], dtype=torch.bool, device="cuda")
            want, w = plain.attend(q[b, i].double()[None], kk, vv, see, see, 128 ** -0.5)
            mass = torch.einsum("htl,lhd->thd", w, vv.abs())[0]
            tol = REL * mass + 2.0 ** -8 * (want[0].abs() + REL * mass) + 1e-6
            assert ((out[b, i].double() - want[0]).abs() <= tol).all()
    assert kvc.get_error(ws) == 0


@pytest.mark.parametrize("layout", ["paged", "ring"])
def test_verification_loop_and_graph(kvc, layout):
    """As a server uses it, in one captured graph: blocks prepared ahead, the draft attended, one of its paths
    appended; then a decode step over the cache equals the same step after kvc_append of those rows."""
    B, H, KV, D, bs, T, P = 2, 8, 2, 64, 16, 8, 4
    paged = layout == "paged"
    d = kvc.make_desc(layout, "none", "bf16", layers=1, batch=B, q_heads=H, kv_heads=KV, head_dim=D,
                      window=0 if paged else 50, block_size=bs if paged else 0, num_blocks=48 if paged else 0,
                      max_blocks_per_seq=24 if paged else 0)
    caches = [kvc.alloc_cache(d, fill=0.0) for _ in range(2)]
    table = torch.randperm(48, generator=torch.Generator().manual_seed(2)).view(2, 24).to(torch.int32).cuda() if paged else None
    ws, other = kvc.alloc_tree_workspace(d, T), kvc.alloc_workspace(d)
    pos = _i32(0, 0)
    parent = _i32(-1, 0, 0, 1, 1, 3, 4, 5, -1, -1, 1, 2, 3, 3, 5, -2).view(2, 8)
    path, n_path = _i32(0, 1, 3, 5, 1, 2, 3, 4).view(2, 4), _i32(4, 2)
    q = torch.empty(B, T, H, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(B, T, KV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.empty_like(q)

    def renew():
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))

    def step():
        kvc.tree_attention(d, caches[0], 0, q, k, v, pos, parent, ws, table, out=out)
        kvc.append_path(d, caches[0], 0, k, v, pos, path, n_path, ws, table)

    renew()
    step()
    caches[0].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = [0, 0]
    for it in range(40):
        renew()
        graph.replay()
        for b, toks in enumerate(([0, 1, 3, 5], [1, 2])):
            # the last token of the path, decoded over a cache that holds the tokens before it
            for tok in toks:
                one = _i32(-10 ** 6, -10 ** 6)
                one[b] = lens[b]
                kvc.append(d, caches[1], 0, k[:, tok].contiguous(), v[:, tok].contiguous(), one, other, block_table=table)
                if it % 9 == 0:
                    ref = kvc.decode_attention(d, caches[1], 0, q[:, tok].contiguous(), one, other, block_table=table)
                    assert float((ref[b].float() - out[b, tok].float()).abs().max()) < 6e-2
                lens[b] += 1
        pos.add_(n_path)
        if paged:
            assert torch.equal(caches[0], caches[1])
    assert torch.equal(caches[0], caches[1])
    assert pos.tolist() == lens and kvc.get_error(ws) == 0


def test_calls_at_once_on_two_streams(kvc):
    runs = [Draft(kvc, "paged", [900, 700, 655, 40], 16, _mixed(16, 4)),
            Draft(kvc, "ring", [2100, 2060], 30, _mixed(30, 2), window=1000, H=16)]
    want = [r.run(kvc) for r in runs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for r, s, o in zip(runs, streams, outs):
            kvc.tree_attention(r.c.d, r.c.cache, r.c.layer, r.q, r.k, r.v, r.pos0, r.parent, r.ws, r.c.table, out=o, stream=s)
    torch.cuda.synchronize()
    for r, w, o in zip(runs, want, outs):
        assert torch.equal(o, w) and kvc.get_error(r.ws) == 0


@pytest.mark.parametrize("layout,D,T,lens", [("paged", 128, 64, [60001]), ("paged", 64, 64, [30000, 9000]),
                                             ("paged", 256, 40, [20000]), ("ring", 128, 32, [5000] * 8)])
def test_many_launches(kvc, layout, D, T, lens):
    """No wait of a role is ever overtaken by the phase after the one it asks for: thousands of launches, each with the
    first one's bits and without an error (one in some hundred long drafts would wait for good)."""
    kw = dict(bs=16) if layout == "paged" else dict(window=4096)
    s = Draft(kvc, layout, lens, T, [_tree(T, "random", b) for b in range(len(lens))], H=32 if layout == "ring" else 8,
              KV=8 if layout == "ring" else 2, D=D, **kw)
    first = s.run(kvc, calls=1).view(torch.int16).clone()
    c, out = s.c, torch.empty_like(s.q)
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(4000):
        kvc.tree_attention(c.d, c.cache, c.layer, s.q, s.k, s.v, s.pos0, s.parent, s.ws, c.table, out=out)
        same &= (out.view(torch.int16) == first).all()
    assert kvc.get_error(s.ws) == 0 and bool(same)
