"""kvc_decode_attention_shared on the GPU against the formula in float64, whatever the groups say.

Tolerance as for the scored prefill (tests/test_gpu_scored.py): a weight's base-2 argument is rounded
to fp16 (ln 2 2^-7 in numerator and denominator, the fp16 result 2^-11 twice) and the weight to bf16
(2^-8); fp32 statistics 1e-3; the output to bf16."""

import math

import pytest
import torch

from tests import plain_ops as plain
from tests.cache_builder import Built

pytestmark = pytest.mark.gpu

REL = 2.0 ** -8 + 1.3e-2


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _tables(lens, prefix, bs, spare=0):
    """Physical blocks of each sequence: `prefix` [(members, blocks)] shared, the rest private; scattered."""
    need = [-(-n // bs) for n in lens]
    total = sum(need) + sum(nb for _, nb in prefix) + spare
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(len(lens) * 31 + bs)).tolist()
    tables = [[] for _ in lens]
    for members, nb in prefix:
        blocks = [perm.pop() for _ in range(nb)]
        for b in members:
            tables[b] = blocks[:need[b]]
    for b, n in enumerate(need):
        while len(tables[b]) < n:
            tables[b].append(perm.pop())
    return tables


def _check(c, out, dead=(), skip=(), rel=REL):
    for b, n in enumerate(c.lens):
        if b in skip:
            continue
        ps = [p for p in range(n) if int(c.table[b, p // c.bs]) >= 0 and int(c.table[b, p // c.bs]) not in dead]
        if not ps:
            assert not out[b].any()
            continue
        k, v = c.rows(b, ps)
        see = torch.ones(1, len(ps), dtype=torch.bool, device="cuda")
        q = c.q[b].double()
        if getattr(c, "baked", False):
            q = plain.rotate(q, torch.tensor(n - 1, device="cuda"), plain.frequencies(c.D)[0], 1.0, "half")
        want, w = plain.attend(q[None], k, v, torch.zeros(1, len(ps), device="cuda"), see, c.scale)
        weight = torch.einsum("htl,lhd->thd", w, v.abs().repeat_interleave(c.H // c.KV, 1))[0]
        tol = rel * weight + 2.0 ** -8 * (want[0].abs() + rel * weight) + 1e-6
        err = (out[b].double() - want[0]).abs()
        assert torch.isfinite(out[b].float()).all()
        assert (err <= tol).all(), (b, float((err / tol).max()))


def _run(kvc, lens, group, prefix, H=8, KV=2, D=128, bs=16, dead=(), valid=None, calls=2, tables=None, **kw):
    tables = _tables(lens, prefix, bs) if tables is None else tables
    c = Built(kvc, "paged", "bf16", lens, H, KV, D, bs=bs, tables=tables, qstd=1.5, **kw)
    ws = kvc.alloc_shared_workspace(c.d)
    gt = torch.tensor(group, dtype=torch.int32, device="cuda")
    vb = None
    if dead:
        mask = torch.ones(c.d.num_blocks, dtype=torch.bool)
        mask[list(dead)] = False
        vb = kvc.pack_valid_bits(mask).cuda()
    out = torch.empty_like(c.q)
    first = None
    for _ in range(calls):
        out.fill_(float("nan"))
        kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, gt, ws, c.table, valid_bits=vb, out=out)
        assert first is None or torch.equal(first, out)      # the same sums in the same order
        first = out.clone()
    _check(c, out, dead)
    return c, ws, gt, out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_head_dims_and_blocks(kvc, D, bs):
    lens = [400, 290, 333, 257, 310, 41, 275]
    _, ws, _, _ = _run(kvc, lens, [0, 0, 1, 1, 1, -1, 1], [((0, 1), 256 // bs), ((2, 3, 4, 6), 256 // bs)], D=D, bs=bs)
    assert kvc.get_error(ws) == 0


@pytest.mark.parametrize("H,KV", [(1, 1), (2, 2), (3, 1), (10, 2), (16, 1), (14, 2), (128, 1), (4, 4)])
@pytest.mark.parametrize("n", [2, 9])
def test_head_groups_and_members(kvc, H, KV, n):
    _run(kvc, [130 + 7 * i for i in range(n)], [0] * n, [(range(n), 8)], H=H, KV=KV)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_columns_of_several_tiles(kvc, D):
    """More members x heads than one Q tile, two, and a column's worth; some prefix tiles partly filled."""
    for n, H in ((17, 8), (33, 8), (70, 8), (130, 1)):
        lens = [100 + i % 40 for i in range(n)]
        _run(kvc, lens, [0] * n, [(range(n), 11)], H=H, KV=1, bs=8, D=D)


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 9, 63])
def test_prefix_lengths(kvc, blocks):
    """From one block to many; 16-row blocks against 64-key tiles."""
    lens = [blocks * 16 + 1 + 5 * i for i in range(4)]
    _run(kvc, lens, [2, 2, 2, 2], [(range(4), blocks)])


def test_long_prefix_many_shares(kvc):
    n = 5
    _run(kvc, [6000 + 100 * i for i in range(n)], [1] * n, [(range(n), 370)], H=8, KV=2)
    _run(kvc, [6000 + 100 * i for i in range(n)], [1] * n, [(range(n), 370)], H=2, KV=1, D=64)


def test_mixed_group_lists(kvc):
    """Ids out of order, singles, members apart, two groups on one prefix, several groups, an id
    past the batch (reported; that sequence counts as alone)."""
    lens = [200, 150, 170, 129, 300, 140, 222, 131, 160]
    pre = [((0, 4, 6), 8), ((1, 2, 8), 8), ((3, 5, 7), 8)]
    _, ws, _, _ = _run(kvc, lens, [8, 3, 3, -5, 8, -1, 8, 0, 3], pre)
    assert kvc.get_error(ws) == 0
    _, ws, _, _ = _run(kvc, lens, [5, 3, 3, 1, 5, 1, 5, 1, 9], pre)
    assert kvc.get_error(ws) == kvc.KVC_DEV_BAD_ENTRY
    _run(kvc, lens, [-1] * 9, pre)
    _run(kvc, lens, [4] * 9, pre)              # one group whose tables have nothing in common
    _run(kvc, lens, [0, 1, 2, 3, 4, 5, 6, 7, 8], pre)


def test_short_members_and_ends(kvc):
    """A member that ends inside the prefix limits what is shared; one that ends with it has no
    rows of its own; tables that part early."""
    bs = 16
    _run(kvc, [200, 50, 170], [0, 0, 0], [((0, 1, 2), 8)])
    _run(kvc, [200, 3, 170], [0, 0, 0], [((0, 1, 2), 8)])
    _run(kvc, [128, 128, 128], [0, 0, 0], [((0, 1, 2), 8)])
    _run(kvc, [128, 112, 129, 127], [0, 0, 0, 0], [((0, 1, 2, 3), 8)])
    t = _tables([160, 160, 160], [((0, 1, 2), 10)], bs, spare=2)
    t[2] = t[2][:3] + [max(max(x) for x in t) + 1] + t[2][4:]     # its fourth block is its own
    _run(kvc, [160, 160, 160], [0, 0, 0], None, tables=t)


@pytest.mark.parametrize("bs", [8, 16, 64])
def test_absent_blocks(kvc, bs):
    """Blocks of the prefix that are not resident, or mapped by nobody, are not attended."""
    lens = [400, 380, 450]
    pre = 256 // bs
    t = _tables(lens, [((0, 1, 2), pre)], bs)
    dead = [t[0][0], t[0][2], t[0][pre - 1], t[1][-1]]
    _run(kvc, lens, [0, 0, 0], None, bs=bs, tables=t, dead=dead)
    _run(kvc, lens, [0, 0, 0], None, bs=bs, tables=t, dead=t[0][:pre])          # the whole prefix
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 128, bs=bs, tables=t, qstd=1.5)
    c.table[:, 1] = -1
    if pre > 4:
        c.table[:, 3:5] = -1
    ws = kvc.alloc_shared_workspace(c.d)
    gt = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, gt, ws, c.table)
    _check(c, out)
    assert kvc.get_error(ws) == 0


def test_bad_block_in_the_prefix_is_reported(kvc):
    lens = [100, 90]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 128, tables=_tables(lens, [((0, 1), 4)], 16), qstd=1.5)
    c.table[:, 2] = c.d.num_blocks + 5
    ws = kvc.alloc_shared_workspace(c.d)
    gt = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, gt, ws, c.table)
    assert kvc.get_error(ws) == kvc.KVC_DEV_BAD_BLOCK
    _check(c, out, dead=(c.d.num_blocks + 5,))


def test_many_sequences(kvc):
    """More sequences than a plan thread block's width, in many groups."""
    n = 300
    lens = [33 + (i * 13) % 50 for i in range(n)]
    members = [[b for b in range(n) if b % 37 == k] for k in range(37)]
    _run(kvc, lens, [b % 37 for b in range(n)], [(m, 2) for m in members], H=4, KV=1, D=64)


def test_one_sequence_and_split_counts(kvc):
    _run(kvc, [300], [0], [((0,), 4)])
    for ns in (1, 3, 40):
        _run(kvc, [300, 290, 280], [0, 0, 0], [((0, 1, 2), 16)], num_splits=ns)


def test_baked_rope(kvc):
    """Each member's query is rotated at its own position, in both parts."""
    lens = [150, 131, 200]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 64, tables=_tables(lens, [((0, 1, 2), 8)], 16), rope="baked", qstd=1.0)
    c.baked = True
    ws = kvc.alloc_shared_workspace(c.d)
    gt = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, gt, ws, c.table)
    # the rotated (and, for the sequences' own keys, scaled) query is rounded to bf16: scores off by
    # 2^-8 sum |q_i k_i| scale, twice in a weight
    qk = max(float(torch.einsum("hd,lhd->hl", c.q[b].double().abs(),
                                c.rows(b, range(n))[0].abs().repeat_interleave(4, 1)).amax())
             for b, n in enumerate(lens)) * c.scale
    _check(c, out, rel=REL + math.expm1(2 * 2.0 ** -8 * qk))


def test_equals_plain_decode_and_shares_its_workspace(kvc):
    lens = [500, 470, 610, 333]
    c, ws, gt, out = _run(kvc, lens, [0, 0, 0, 0], [(range(4), 18)])
    for _ in range(2):
        ref = kvc.decode_attention(c.d, c.cache, c.layer, c.q, c.pos, ws, block_table=c.table)
        assert float((ref.float() - out.float()).abs().max()) < 6e-2
        again = kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, gt, ws, c.table)
        assert torch.equal(again, out)


def test_block_share_append_and_graph(kvc):
    """As a server uses it: a prompt in one sequence's blocks, shared by kvc_block_share, then steps
    (block_prepare, append with norms and rotation, shared attention) captured in one graph and
    replayed while positions advance; against plain decode attention on the same cache."""
    B, H, KV, D, bs = 4, 8, 2, 64, 16
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=B, q_heads=H, kv_heads=KV, head_dim=D, block_size=bs,
                      num_blocks=64, max_blocks_per_seq=12)
    cache, ws, state = kvc.alloc_cache(d, fill=float("nan")), kvc.alloc_shared_workspace(d), kvc.BlockState(d)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    qk = kvc.make_qk(d, kvc.make_rotary("half", dim=D), eps=1e-5)
    n0 = 70
    for p in range(n0):
        kvc.block_prepare(d, cache, i32(p, -1, -1, -1), state, ws)
    x = torch.randn(B, n0, H + 2 * KV, D, device="cuda").to(torch.bfloat16)
    kvc.append_qk(d, cache, 0, x[:, :, :H], x[:, :, H:H + KV], x[:, :, H + KV:], i32(0, 0, 0, 0), ws, qk,
                  n_tok=i32(n0, 0, 0, 0), block_table=state.table)
    kvc.block_share(d, state, i32(0, 0, 0), i32(1, 2, 3), i32(5, 5, 5), ws)
    assert kvc.get_error(ws) == 0
    pos, group = i32(n0, n0, n0, n0), i32(0, 0, 0, 0)
    new = torch.empty(B, H + 2 * KV, D, dtype=torch.bfloat16, device="cuda")
    q, out = (torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        kvc.block_prepare(d, cache, pos, state, ws)
        kvc.append_qk(d, cache, 0, new[:, :H], new[:, H:H + KV], new[:, H + KV:], pos, ws, qk,
                      block_table=state.table, q_out=q)
        kvc.decode_attention_shared(d, cache, 0, q, pos, group, ws, state.table, valid_bits=state.valid_bits, out=out)

    new.copy_(torch.randn(new.shape, device="cuda"))
    step()                                       # position n0: every sequence copies the shared last block
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = kvc.alloc_workspace(d)
    for _ in range(30):
        pos.add_(1)
        new.copy_(torch.randn(new.shape, device="cuda"))
        graph.replay()
        ref = kvc.decode_attention(d, cache, 0, q, pos, other, block_table=state.table, valid_bits=state.valid_bits)
        assert float((ref.float() - out.float()).abs().max()) < 6e-2
    assert kvc.get_error(ws) == 0
    assert len({int(x) for x in state.table[:, 0]}) == 1 and len({int(x) for x in state.table[:, 4]}) == 4


def test_offsets_past_32_bits(kvc):
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=3, q_heads=8, kv_heads=8, head_dim=128, block_size=16,
                      num_blocks=140000, max_blocks_per_seq=6)
    cache = kvc.alloc_cache(d)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.tensor([[139999, 5, 70000, 139990, 1, 2], [139999, 5, 70000, 139990, 139991, 3],
                          [139999, 5, 70000, 139990, 139992, 139993]], dtype=torch.int32, device="cuda")
    for blk in table.flatten().unique().tolist():
        cache[0, :, blk] = torch.randn(2, 8, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(3, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.tensor([70, 80, 95], dtype=torch.int32, device="cuda")
    ws = kvc.alloc_shared_workspace(d)
    out = kvc.decode_attention_shared(d, cache, 0, q, pos, torch.zeros(3, dtype=torch.int32, device="cuda"), ws, table)
    score = kvc.decode_attention_scored(d, cache, 0, q, pos, ws, kvc.make_score(), block_table=table)
    for b in range(3):
        n = int(pos[b]) + 1
        rows = cache[0, :, table[b].long()].double()             # [2, 6, 8, 16, 128]
        k, v = (rows[i].permute(0, 2, 1, 3).reshape(96, 8, 128)[:n] for i in range(2))
        see = torch.ones(1, n, dtype=torch.bool, device="cuda")
        want, w = plain.attend(q[b].double()[None], k, v, see, see, 128 ** -0.5)
        weight = torch.einsum("htl,lhd->thd", w, v.abs())[0]
        for got in (out, score):
            tol = REL * weight + 2.0 ** -8 * (want[0].abs() + REL * weight) + 1e-6
            assert ((got[b].double() - want[0]).abs() <= tol).all()
    assert kvc.get_error(ws) == 0


def test_calls_at_once_on_two_streams(kvc):
    """Each with its own workspace: the results of the calls alone."""
    runs = [_run(kvc, [900, 700, 655, 40, 333], [0, 0, 0, 1, 1], [(range(3), 40), ((3, 4), 2)]),
            _run(kvc, [2100, 2060], [1, 1], [(range(2), 128)], H=16)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(r[3]) for r in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, ws, gt, _), s, o in zip(runs, streams, outs):
            kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, gt, ws, c.table, out=o, stream=s)
    torch.cuda.synchronize()
    for (c, ws, gt, want), o in zip(runs, outs):
        assert torch.equal(o, want)
        assert kvc.get_error(ws) == 0
