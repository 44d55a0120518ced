"""Block weights and eviction on the GPU.

Weights against float64: a score is an fp32 sum of D products (D 2^-24 of sum |q_i k_i| scale, in numerator and
denominator of a weight), an exponential 2^-22, and the sums over heads and rows are fp32.  Outputs as for the
selected decode.  Evictions are whole numbers and have to be equal."""

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


def _check(c, out, weights, base, decay, dead=(), skip=(), q=None, rel=REL, more=0.0):
    G = c.H // c.KV
    for b, n in enumerate(c.lens):
        if b in skip:
            continue
        ps = [p for p in range(n) if 0 <= int(c.table[b, p // c.bs]) < c.d.num_blocks
              and int(c.table[b, p // c.bs]) not in dead]
        want_w = base[b].double() * decay if decay else torch.zeros_like(base[b]).double()
        add = torch.zeros_like(want_w)
        if ps:
            k, v = c.rows(b, ps)
            lb = torch.tensor([p // c.bs for p in ps], device="cuda")
            qk = 0.0
            for h in range(c.KV):
                qq = (c.q if q is None else q)[b, h * G:h * G + G].double()
                want, w = part.attend(qq, k[:, h], v[:, h], c.scale)
                add.index_add_(0, lb, w.sum(0))
                qk = max(qk, float((qq.abs() @ k[:, h].abs().T).max()) * c.scale)
                o, mass = out[b, h * G:h * G + G].double(), w @ v[:, h].abs()
                tol = rel * mass + 2.0 ** -8 * (want.abs() + rel * mass) + 1e-6
                assert ((o - want).abs() <= tol).all(), (b, h, float(((o - want).abs() / tol).max()))
            near = math.expm1(2 * c.D * 2.0 ** -24 * qk) + (c.H + c.bs + 64) * 2.0 ** -24 + 2.0 ** -20 + more
        else:
            assert not out[b].any()
            near = 0.0
        got = weights[b].double()
        err = (got - (want_w + add)).abs()
        tol = near * add + 2.0 ** -23 * want_w.abs() + 1e-7
        assert torch.isfinite(got).all()
        assert (err <= tol).all(), (b, float((err / tol).max()))


def _run(kvc, lens, H=8, KV=2, D=128, bs=16, dtype="bf16", decay=0.5, calls=2, absent=(), dead=(), num_splits=0, **kw):
    c = Built(kvc, "paged", dtype, lens, H, KV, D, bs=bs, num_splits=num_splits, qstd=1.5, **kw)
    for b, lb in absent:
        c.table[b, lb] = -1
    vb, gone = None, ()
    if dead:
        gone = [int(c.table[b, lb]) for b, lb in dead]
        mask = torch.ones(c.d.num_blocks, dtype=torch.bool)
        mask[gone] = False
        vb = kvc.pack_valid_bits(mask).cuda()
    ws = kvc.alloc_weighed_workspace(c.d)
    base = torch.rand(c.table.shape, device="cuda") * 5
    weights = base.clone()
    if decay == 0.0:
        weights.fill_(float("nan"))                    # the old values are not read
    first = weights.clone()
    seen = None
    for _ in range(calls):
        weights.copy_(first)
        out = kvc.decode_attention_weighed(c.d, c.cache, c.layer, c.q, c.pos, weights, ws, c.table, valid_bits=vb,
                                           decay=decay)
        assert seen is None or (torch.equal(seen[0], out) and torch.equal(seen[1], weights))
        seen = (out, weights.clone())
    _check(c, out, weights, base, decay, dead=gone)
    assert kvc.get_error(ws) == 0
    return c, ws, base, out, weights


@pytest.mark.parametrize("dtype,D,H,KV,bs", [
    ("bf16", 128, 8, 2, 16), ("bf16", 64, 3, 1, 8), ("bf16", 256, 16, 1, 12), ("bf16", 64, 4, 4, 5),
    ("bf16", 128, 10, 2, 100), ("bf16", 64, 2, 2, 300), ("bf16", 256, 8, 8, 64), ("i8", 128, 8, 4, 4),
    ("i8", 256, 6, 2, 8), ("i8", 128, 4, 1, 64), ("bf16", 128, 128, 1, 16), ("bf16", 64, 1, 1, 1)])
@pytest.mark.parametrize("decay", [0.0, 0.9, 1.0])
def test_shapes(kvc, dtype, D, H, KV, bs, decay):
    _run(kvc, [1, 5 * bs, 11 * bs + (3 if bs > 3 else 0), 30 * bs - 1], H, KV, D, bs, dtype, decay)


@pytest.mark.parametrize("dtype", ["bf16", "i8"])
@pytest.mark.parametrize("ns", [0, 1, 7, 300])
def test_splits(kvc, dtype, ns):
    """Shares that end inside blocks and sub-tiles."""
    _run(kvc, [3333, 17, 1200, 700], dtype=dtype, num_splits=ns)
    _run(kvc, [3333], dtype=dtype, num_splits=ns, H=4, KV=4)


def test_absent_blocks(kvc):
    _run(kvc, [300, 200, 250, 30], absent=[(0, 0), (0, 5), (2, 15), (3, 0), (3, 1)], dead=[(1, 3), (1, 12), (2, 4)])
    _run(kvc, [400], absent=[(0, 3), (0, 4)], dead=[(0, 20)])


def test_many_sequences_and_long_tables(kvc):
    _run(kvc, [33 + (i * 13) % 50 for i in range(150)], H=4, KV=1, D=64, bs=8)
    _run(kvc, [70000], H=2, KV=1, D=64, bs=8)                # more blocks than the decode plans by itself


def test_idle_and_past_the_table(kvc):
    """A sequence without a position decays and gets zeros; one past the table attends the table."""
    lens = [150, 131, 96]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 64, qstd=1.5)
    ws = kvc.alloc_weighed_workspace(c.d)
    base = torch.rand(c.table.shape, device="cuda")
    weights = base.clone()
    out = kvc.decode_attention_weighed(c.d, c.cache, c.layer, c.q, _i32(149, -1, 10 ** 9), weights, ws, c.table, decay=0.25)
    assert kvc.get_error(ws) == kvc.KVC_DEV_BAD_POSITION
    assert not out[1].any() and torch.equal(weights[1], base[1] * 0.25)
    _check(c, out, weights, base, 0.25, skip=(1, 2))


def test_bad_block(kvc):
    c = Built(kvc, "paged", "bf16", [100, 90], 8, 2, 128, qstd=1.5)
    c.table[0, 2] = c.d.num_blocks + 3
    ws = kvc.alloc_weighed_workspace(c.d)
    base = torch.zeros(c.table.shape, device="cuda")
    weights = base.clone()
    out = kvc.decode_attention_weighed(c.d, c.cache, c.layer, c.q, c.pos, weights, ws, c.table)
    assert kvc.get_error(ws) == kvc.KVC_DEV_BAD_BLOCK
    _check(c, out, weights, base, 1.0)


def test_large_scores_and_nan_queries(kvc):
    """One key that takes all the weight: the others' weights underflow to 0, never to anything else; a query that
    is NaN gives NaN, in its own sequence alone."""
    c = Built(kvc, "paged", "bf16", [500, 400], 4, 1, 64, qstd=1.5)
    row = c.kv[0][333]
    c.cache[c.layer, 0, row[0], :, row[1]] = (c.q[0].float().sum(0) * 40).to(torch.bfloat16)
    c.k[c.index[row]] = c.cache[c.layer, 0, row[0], :, row[1]].double()
    ws = kvc.alloc_weighed_workspace(c.d)
    base = torch.zeros(c.table.shape, device="cuda")
    weights = base.clone()
    out = kvc.decode_attention_weighed(c.d, c.cache, c.layer, c.q, c.pos, weights, ws, c.table, decay=0.0)
    _check(c, out, weights, base, 0.0, more=1e-3)
    q = c.q.clone()
    q[1, 2, 5] = float("nan")
    w2 = base.clone()
    out2 = kvc.decode_attention_weighed(c.d, c.cache, c.layer, q, c.pos, w2, ws, c.table, decay=0.0)
    assert torch.equal(out2[0], out[0]) and torch.equal(w2[0], weights[0])
    assert torch.isnan(out2[1, 2]).all() and torch.isnan(w2[1, :400 // 16]).all()


def test_baked_rope(kvc):
    lens = [150, 131]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 64, rope="baked", qstd=1.0)
    ws = kvc.alloc_weighed_workspace(c.d)
    base = torch.zeros(c.table.shape, device="cuda")
    weights = base.clone()
    out = kvc.decode_attention_weighed(c.d, c.cache, c.layer, c.q, c.pos, weights, ws, c.table)
    turned = plain.rotate(c.q.double(), c.pos.double(), plain.frequencies(64)[0], 1.0, "half")
    qk = max(float(torch.einsum("hd,lhd->hl", turned[b].abs(), c.rows(b, range(n))[0].abs().repeat_interleave(4, 1)).amax())
             for b, n in enumerate(lens)) * c.scale
    off = math.expm1(2 * 2.0 ** -8 * qk)                      # the rotated query is rounded to bf16
    _check(c, out, weights, base, 1.0, q=turned, rel=REL + off, more=off)


def test_two_streams(kvc):
    runs = [_run(kvc, [900, 700, 655, 40, 333]), _run(kvc, [2100, 2060], H=16)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(torch.empty_like(r[3]), r[2].clone()) for r in runs]
    torch.cuda.synchronize()
    for _ in range(10):
        for (c, ws, base, _, _), s, (o, w) in zip(runs, streams, got):
            with torch.cuda.stream(s):
                w.copy_(base)
                kvc.decode_attention_weighed(c.d, c.cache, c.layer, c.q, c.pos, w, ws, c.table, decay=0.5, out=o)
    torch.cuda.synchronize()
    for (c, ws, _, out, weights), (o, w) in zip(runs, got):
        assert torch.equal(o, out) and torch.equal(w, weights)
        assert kvc.get_error(ws) == 0


# ---------------------------------------------------------------- eviction
def _evict_state(kvc, B, maxb, nblocks, bs=16, seed=0, share=0, holes=0.1, free=5):
    """A block manager's state with random tables: the first `share` blocks of all sequences in common."""
    g = torch.Generator().manual_seed(seed)
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=B, q_heads=2, kv_heads=1, head_dim=64, block_size=bs,
                      num_blocks=nblocks, max_blocks_per_seq=maxb)
    state = kvc.BlockState(d)
    perm = torch.randperm(nblocks, generator=g).tolist()
    common = [perm.pop() for _ in range(share)]
    table = [[-1] * maxb for _ in range(B)]
    ref = [0] * nblocks
    for b in range(B):
        for lb in range(maxb):
            if float(torch.rand(1, generator=g)) < holes or (lb >= share and len(perm) <= free):
                continue
            table[b][lb] = common[lb] if lb < share else perm.pop()
            ref[table[b][lb]] += 1
    for p in common:
        if ref[p] == 0:
            perm.append(p)
    state.table.copy_(torch.tensor(table, dtype=torch.int32))
    state.refcount.copy_(torch.tensor(ref, dtype=torch.int32))
    stack = perm + [-7] * (nblocks - len(perm))
    state.free_list.copy_(torch.tensor(stack, dtype=torch.int32))
    state.free_count.fill_(len(perm))
    mask = torch.tensor([r > 0 for r in ref])
    state.valid_bits.copy_(kvc.pack_valid_bits(mask))
    return d, state, table, ref, stack, len(perm), mask


def _check_evict(kvc, d, state, weights, pos, keep, first, recent, model, ws=None):
    table, ref, stack, count, mask = model
    ws = kvc.alloc_workspace(d) if ws is None else ws
    w = weights.tolist()
    want_stack, want_count, back = part.evict(w, table, pos, d.block_size, keep, first, recent, ref, stack, count,
                                              d.num_blocks)
    mask = mask.clone()
    mask[back] = False
    kvc.block_evict(d, state, weights, _i32(*pos), keep, ws, first=first, recent=recent)
    assert state.table.tolist() == table
    assert state.refcount.tolist() == ref
    assert int(state.free_count) == want_count
    assert state.free_list.tolist()[:want_count] == want_stack[:want_count]
    assert torch.equal(state.valid_bits.cpu(), kvc.pack_valid_bits(mask))
    assert torch.equal(weights.nan_to_num(nan=-5.0).cpu(), torch.tensor(w).nan_to_num(nan=-5.0))
    return (table, ref, want_stack, want_count, mask), ws


@pytest.mark.parametrize("B,maxb,share", [(1, 1, 0), (1, 40, 0), (3, 33, 4), (7, 130, 0), (2, 3000, 100), (1, 70000, 0)])
@pytest.mark.parametrize("kind", ["random", "quarters", "equal", "special"])
def test_evict(kvc, B, maxb, share, kind):
    bs = 16
    d, state, *model = _evict_state(kvc, B, maxb, B * maxb + 9, bs, seed=B + maxb, share=share)
    w = torch.rand(B, maxb)
    if kind == "quarters":
        w = (w * 4).round() / 4 - 0.5
    elif kind == "equal":
        w.fill_(2.0)
    elif kind == "special":
        pick = torch.arange(B * maxb).view(B, maxb) % 7
        w = torch.where(pick == 0, float("nan"), torch.where(pick == 1, -0.0, torch.where(pick == 2, 0.0, torch.where(
            pick == 3, float("inf"), torch.where(pick == 4, -3.0, torch.where(pick == 5, float("-inf"), w))))))
    weights = w.cuda()
    pos = [maxb * bs - 1 - (b * 7) % max(1, maxb * bs // 3) for b in range(B)]
    keep = max(2, maxb // 2)
    first, recent = (1, 1) if keep < 6 else (2, 4)
    model, ws = _check_evict(kvc, d, state, weights, pos, keep, first, recent, model)
    # again: nothing is left to give back
    model, ws = _check_evict(kvc, d, state, weights, pos, keep, first, recent, model, ws)
    if keep > 4:
        _check_evict(kvc, d, state, weights, pos, keep // 2 + 1, 0, 1, model, ws)
    assert kvc.get_error(ws) == 0


def test_evict_leaves_idle_and_short_sequences(kvc):
    d, state, *model = _evict_state(kvc, 4, 50, 210, holes=0.0)
    weights = torch.rand(4, 50, device="cuda")
    _check_evict(kvc, d, state, weights, [799, -1, 30, 16 * 20], 20, 1, 1, model)


def test_evict_all_sequences_of_a_shared_prefix(kvc):
    """A block goes back once the last sequence that maps it gives it up."""
    d, state, *model = _evict_state(kvc, 5, 20, 120, share=12, holes=0.0)
    weights = torch.rand(5, 20, device="cuda")
    weights[:, :12] = 0.0
    model, ws = _check_evict(kvc, d, state, weights, [319] * 5, 10, 0, 2, model)
    weights.fill_(1.0)
    _check_evict(kvc, d, state, weights, [319] * 5, 3, 0, 2, model, ws)


def test_evict_reports_bad_blocks(kvc):
    d, state, *_ = _evict_state(kvc, 1, 10, 20, holes=0.0)
    state.table[0, 3] = 21
    weights = torch.ones(1, 10, device="cuda")
    weights[0, 3] = 0.0
    ws = kvc.alloc_workspace(d)
    kvc.block_evict(d, state, weights, _i32(159), 9, ws)
    assert kvc.get_error(ws) == kvc.KVC_DEV_BAD_BLOCK
    assert int(state.table[0, 3]) == -1 and int(state.free_count) == 10


@pytest.mark.parametrize("dtype", ["bf16", "i8"])
def test_bounded_cache_loop_and_graph(kvc, dtype):
    """As a server uses it: a cache held to 6 blocks a sequence, each step of two layers prepared, appended, weighed
    and cut back, in one captured graph; against plain decode on the tables as they stand."""
    B, H, KV, D, bs, keep = 2, 4, 2, 128, 8, 6
    d = kvc.make_desc("paged", "none", dtype, layers=2, batch=B, q_heads=H, kv_heads=KV, head_dim=D, block_size=bs,
                      num_blocks=16, max_blocks_per_seq=40)
    cache, state = kvc.alloc_cache(d, fill=float("nan")), kvc.BlockState(d)
    ws, other = kvc.alloc_weighed_workspace(d), kvc.alloc_workspace(d)
    weights = torch.zeros(B, 40, device="cuda")
    pos = _i32(0, 0)
    q = torch.empty(2, B, H, D, dtype=torch.bfloat16, device="cuda")
    kn, vn = (torch.empty(2, B, KV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.empty_like(q)

    def renew():
        for x in (q, kn, vn):
            x.copy_(torch.randn(x.shape, device="cuda"))

    def step():
        kvc.block_prepare(d, cache, pos, state, ws)
        for layer in range(2):
            kvc.append(d, cache, layer, kn[layer], vn[layer], pos, ws, block_table=state.table)
            kvc.decode_attention_weighed(d, cache, layer, q[layer], pos, weights, ws, state.table, state.valid_bits,
                                         decay=0.9 if layer == 0 else 1.0, out=out[layer])

    renew()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    cut = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cut):
        kvc.block_evict(d, state, weights, pos, keep, ws, first=1, recent=2)
    for t in range(1, 300):
        pos.add_(1)
        renew()
        before = weights.clone()
        graph.replay()
        if t % 37 == 0:
            for layer in range(2):
                ref = kvc.decode_attention(d, cache, layer, q[layer], pos, other, block_table=state.table,
                                           valid_bits=state.valid_bits)
                assert float((ref.float() - out[layer].float()).abs().max()) < 6e-2
            # a step adds H to each sequence for each layer
            more = weights.sum(1) - 0.9 * before.sum(1)
            assert float((more - 2 * H).abs().max()) < 1e-3
        cut.replay()
        if t % 37 == 0:
            nb = t // bs + 1
            assert (state.table >= 0).sum(1).tolist() == [min(nb, keep)] * B
            assert int(state.free_count) == 16 - B * min(nb, keep)
            assert (state.table[:, 0] >= 0).all() and (state.table[:, max(0, nb - 2):nb] >= 0).all()
    assert kvc.get_error(ws) == 0
