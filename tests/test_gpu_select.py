"""Block bounds, block selection and decode over selected blocks on the GPU.

Bounds and selections are whole numbers and have to be equal.  Outputs against float64: a weight enters the
second product rounded to bf16 (2^-8 of it; INT8 caches: fp16, less), fp32 scores and statistics leave 1e-3 of
sum w |v| at most, and the output is rounded to bf16 once."""

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


def _value_rows(c, b, ps):
    """Key rows [len, KV, D] fp32 as the library reads them."""
    return c.rows(b, ps)[0].float()


def _bounds(kvc, c, first, n, n_new=None, ws=None, bounds=None):
    bounds = kvc.alloc_bounds(c.d) if bounds is None else bounds
    kvc.block_bounds(c.d, c.cache, c.layer, bounds, _i32(*first), max(n) if n_new is None else n_new,
                     c.ws if ws is None else ws, c.table, n_tok=_i32(*n))
    return bounds


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 128), ("f32", 256), ("bf16", 64), ("bf16", 128),
                                     ("bf16", 256), ("i8", 128), ("i8", 256)])
@pytest.mark.parametrize("bs", [4, 16, 20, 64])
def test_bounds_of_a_prompt(kvc, dtype, D, bs):
    """Every block of ragged sequences, the last one partly filled (garbage behind)."""
    lens = [1, bs, bs + 1, 3 * bs - 1, 150]
    c = Built(kvc, "paged", dtype, lens, 6, 3, D, bs=bs, seed=bs)
    bounds = _bounds(kvc, c, [0] * 5, lens)
    codes, steps = kvc.bounds_views(c.d, bounds)
    for b, n in enumerate(lens):
        for lb in range(-(-n // bs)):
            k = _value_rows(c, b, range(lb * bs, min(n, lb * bs + bs)))
            for h in range(3):
                want, step = part.ends(k[:, h])
                at = int(c.table[b, lb])
                assert torch.equal(codes[c.layer, at, h], want), (b, lb, h)
                assert float(steps[c.layer, at, h]) == float(step)
                # and they bound the keys from outside, up to the rounding of a step
                top = codes[c.layer, at, h].double() * steps[c.layer, at, h].double()
                slack = 2.0 ** -22 * float(step) * 127
                assert (k[:, h].double() <= top[0] + slack).all() and (k[:, h].double() >= top[1] - slack).all()
    assert kvc.get_error(c.ws) == 0


def test_bounds_of_a_step_leave_the_other_blocks(kvc):
    lens = [40, 33, 32, 7]
    c = Built(kvc, "paged", "bf16", lens, 4, 2, 64, bs=16)
    bounds = kvc.alloc_bounds(c.d)
    bounds.fill_(85)
    before = bounds.clone()
    # one token each, a sequence without one, one in front of position 0 and one past it
    kvc.block_bounds(c.d, c.cache, c.layer, bounds, _i32(39, 32, 31, -1), 1, c.ws, c.table)
    codes, steps = kvc.bounds_views(c.d, bounds)
    old, _ = kvc.bounds_views(c.d, before)
    touched = [(b, (n - 1) // 16) for b, n in enumerate(lens[:3])]
    for b, lb in touched:
        k = _value_rows(c, b, range(lb * 16, lens[b]))
        for h in range(2):
            want, step = part.ends(k[:, h])
            assert torch.equal(codes[c.layer, int(c.table[b, lb]), h], want)
    same = torch.ones(c.d.num_blocks, dtype=torch.bool)
    same[[int(c.table[b, lb]) for b, lb in touched]] = False
    assert torch.equal(codes[c.layer][same.cuda()], old[c.layer][same.cuda()])
    assert torch.equal(codes[0], old[0])                          # the other layer
    # left padding: positions -3 .. 2 are positions 0 .. 2
    bounds = _bounds(kvc, c, [-3, 0, 0, 0], [6, 0, 0, -4])
    codes, _ = kvc.bounds_views(c.d, bounds)
    assert torch.equal(codes[c.layer, int(c.table[0, 0]), 1], part.ends(_value_rows(c, 0, range(3))[:, 1])[0])
    assert int((kvc.bounds_views(c.d, bounds)[1] != 0).sum()) == 2
    assert kvc.get_error(c.ws) == 0


def test_bounds_errors(kvc):
    c = Built(kvc, "paged", "bf16", [40, 33], 4, 2, 64, bs=16)
    reach = c.table.shape[1] * 16
    _bounds(kvc, c, [reach - 1, 0], [3, 1])
    assert kvc.get_error(c.ws) & kvc.KVC_DEV_BAD_POSITION
    c.table[0, 1] = -1
    bounds = _bounds(kvc, c, [0, 0], [40, 33])
    assert kvc.get_error(c.ws) == kvc.KVC_DEV_UNMAPPED_APPEND
    assert torch.equal(kvc.bounds_views(c.d, bounds)[0][c.layer, int(c.table[0, 2]), 0],
                       part.ends(_value_rows(c, 0, range(32, 40))[:, 0])[0])
    c.table[0, 1] = c.d.num_blocks
    _bounds(kvc, c, [0, 0], [40, 33])
    assert kvc.get_error(c.ws) == kvc.KVC_DEV_BAD_BLOCK
    # positions at the end of int32
    _bounds(kvc, c, [2 ** 31 - 1, 2 ** 31 - 2], [5, 5])
    assert kvc.get_error(c.ws) == kvc.KVC_DEV_BAD_POSITION


def _want_select(kvc, c, bounds, k, first, recent, dead=(), q=None):
    codes, steps = (x[c.layer] for x in kvc.bounds_views(c.d, bounds))
    out = []
    for b, n in enumerate(c.lens):
        nb = -(-n // c.bs)
        row = [int(x) for x in c.table[b, :nb]]
        cand = [lb for lb, x in enumerate(row) if 0 <= x and x not in dead]
        at = torch.tensor([max(x, 0) for x in row] or [0], device="cuda")
        out.append(part.select(codes[at].cpu(), steps[at].cpu(), (c.q if q is None else q)[b].cpu(), cand, nb, k, first,
                               recent, c.H // c.KV))
    return out


def _check_select(c, got, want, k):
    for b, lists in enumerate(want):
        for h, x in enumerate(lists):
            assert got[b, h].tolist() == x + [-1] * (k - len(x)), (b, h)


@pytest.mark.parametrize("dtype,D,H,KV,bs", [("bf16", 128, 8, 2, 16), ("bf16", 64, 3, 1, 8), ("bf16", 256, 16, 1, 12),
                                             ("f32", 128, 4, 4, 16), ("f32", 64, 10, 2, 32), ("i8", 128, 8, 4, 4),
                                             ("i8", 256, 6, 2, 8), ("bf16", 128, 128, 1, 16)])
@pytest.mark.parametrize("k,first,recent", [(1, 0, 1), (3, 1, 1), (7, 0, 2), (40, 2, 3)])
def test_select(kvc, dtype, D, H, KV, bs, k, first, recent):
    lens = [1, 5 * bs, 11 * bs + 3, 30 * bs - 1]
    c = Built(kvc, "paged", dtype, lens, H, KV, D, bs=bs, seed=k)
    c.table[3, 4:9] = -1                                        # given back earlier
    bounds = _bounds(kvc, c, [0, 0, 0, 0], [1, 5 * bs, 11 * bs + 3, 4 * bs])
    bounds = _bounds(kvc, c, [0, 0, 0, 9 * bs], [0, 0, 0, 21 * bs - 1], bounds=bounds)
    ws = kvc.alloc_select_workspace(c.d, k)
    dead = [int(c.table[3, 12]), int(c.table[2, 2])]
    mask = torch.ones(c.d.num_blocks, dtype=torch.bool)
    mask[dead] = False
    bits = kvc.pack_valid_bits(mask).cuda()
    for vb, gone in ((None, ()), (bits, dead)):
        got = kvc.select_blocks(c.d, bounds, c.layer, c.q, c.pos, k, ws, c.table, first=first, recent=recent,
                                valid_bits=vb)
        _check_select(c, got, _want_select(kvc, c, bounds, k, first, recent, gone), k)
    assert kvc.get_error(ws) == 0


def test_select_ties_and_zero_queries(kvc):
    """Blocks alike in their bounds, and a query of zeros: the lowest numbers."""
    lens = [16 * 40, 16 * 21]
    c = Built(kvc, "paged", "bf16", lens, 4, 2, 128)
    bounds = kvc.alloc_bounds(c.d)
    codes, steps = kvc.bounds_views(c.d, bounds)
    codes.fill_(3)
    steps.fill_(0.5)
    codes[c.layer, int(c.table[0, 30]), 1] = 4
    ws = kvc.alloc_select_workspace(c.d, 9)
    q = c.q.abs()
    got = kvc.select_blocks(c.d, bounds, c.layer, q, c.pos, 9, ws, c.table, first=1, recent=2)
    assert got[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 38, 39]
    assert got[0, 1].tolist() == [0, 1, 2, 3, 4, 5, 30, 38, 39]
    got = kvc.select_blocks(c.d, bounds, c.layer, torch.zeros_like(q), c.pos, 9, ws, c.table, first=1, recent=2)
    assert got[1, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 19, 20]
    # negative scores: all channels of q below 0 meet the smaller code; -0 and 0 count the same
    codes[:, :, :, 0] = 0
    codes[:, :, :, 1] = -1
    codes[c.layer, int(c.table[0, 7]), :, 0] = -1
    got = kvc.select_blocks(c.d, bounds, c.layer, q, c.pos, 5, ws, c.table, first=0, recent=1)
    assert got[0, 0].tolist() == [0, 1, 2, 3, 39]
    assert kvc.get_error(ws) == 0


def test_select_many_blocks(kvc):
    """More blocks than one pass of the search holds, k beyond a pass of the lists, and scores that differ in low
    bits alone."""
    n, bs, D = 1531, 4, 64
    c = Built(kvc, "paged", "bf16", [n * bs - 2], 2, 1, D, bs=bs)
    bounds = _bounds(kvc, c, [0], [n * bs - 2])
    for k in (1, 300, 700, 1530, 1531, 2000):
        ws = kvc.alloc_select_workspace(c.d, k)
        got = kvc.select_blocks(c.d, bounds, c.layer, c.q, c.pos, k, ws, c.table, first=0, recent=1)
        _check_select(c, got, _want_select(kvc, c, bounds, k, 0, 1), k)
    codes, steps = kvc.bounds_views(c.d, bounds)
    codes.fill_(1)
    steps[c.layer] = 1.0 + torch.randint(0, 90, steps[c.layer].shape, device="cuda") * 2.0 ** -23
    ws = kvc.alloc_select_workspace(c.d, 100)
    got = kvc.select_blocks(c.d, bounds, c.layer, c.q, c.pos, 100, ws, c.table, first=3, recent=5)
    _check_select(c, got, _want_select(kvc, c, bounds, 100, 3, 5), 100)


def test_select_baked_rotates_the_query(kvc):
    """Blocks whose ends follow the signs of the rotated query (100 of every code: more than any other sum below)
    are chosen before those that follow the query as it came (40 of every code, at most)."""
    c = Built(kvc, "paged", "bf16", [16 * 30], 4, 2, 64)
    bounds = kvc.alloc_bounds(c.d)
    codes, steps = kvc.bounds_views(c.d, bounds)
    steps.fill_(0.25)
    turned = plain.rotate(c.q.double(), c.pos.double(), plain.frequencies(64)[0], 1.0, "half")
    for lb in range(1, 29):
        at = int(c.table[0, lb])
        for h in range(2):
            follow = turned[0, 2 * h] if lb % 4 == 2 else c.q[0, 2 * h].double()
            codes[c.layer, at, h] = (torch.sign(follow) * (100 if lb % 4 == 2 else 40)).to(torch.int8)
    ws = kvc.alloc_select_workspace(c.d, 9)
    for rope, want in (("baked", [0, 2, 6, 10, 14, 18, 22, 26, 29]), ("none", None)):
        d = kvc.make_desc("paged", rope, "bf16", layers=2, batch=1, q_heads=4, kv_heads=2, head_dim=64, block_size=16,
                          num_blocks=c.d.num_blocks, max_blocks_per_seq=c.table.shape[1])
        got = kvc.select_blocks(d, bounds, c.layer, c.q, c.pos, 9, ws, c.table)[0].tolist()
        assert (got == [want, want]) == (rope == "baked")
    assert kvc.get_error(ws) == 0


def test_select_idle_and_bad(kvc):
    lens = [100, 90, 80]
    c = Built(kvc, "paged", "bf16", lens, 4, 2, 64)
    bounds = _bounds(kvc, c, [0] * 3, lens)
    ws = kvc.alloc_select_workspace(c.d, 4)
    pos = _i32(99, -1, 10 ** 6)
    c.table[0, 3] = c.d.num_blocks + 1
    got = kvc.select_blocks(c.d, bounds, c.layer, c.q, pos, 4, ws, c.table)
    assert kvc.get_error(ws) == kvc.KVC_DEV_BAD_POSITION | kvc.KVC_DEV_BAD_BLOCK
    assert (got[1] == -1).all() and 3 not in got[0].tolist()[0]
    assert all(x < c.table.shape[1] for x in got[2].flatten().tolist())


# ---------------------------------------------------------------- attention over lists
def _check_out(c, out, lists, skip=(), rel=REL, q=None):
    """lists[b][h]: the logical blocks attended."""
    G = c.H // c.KV
    for b, n in enumerate(c.lens):
        if b in skip:
            continue
        for h in range(c.KV):
            ps = [p for lb in lists[b][h] for p in range(lb * c.bs, min(n, lb * c.bs + c.bs))]
            o = out[b, h * G:h * G + G].double()
            if not ps:
                assert not o.any()
                continue
            k, v = c.rows(b, ps)
            qq = (c.q if q is None else q)[b, h * G:h * G + G].double()
            want, w = part.attend(qq, k[:, h], v[:, h], c.scale)
            mass = w @ v[:, h].abs()
            tol = rel * mass + 2.0 ** -8 * (want.abs() + rel * mass) + 1e-6
            assert torch.isfinite(o).all()
            assert ((o - want).abs() <= tol).all(), (b, h, float(((o - want).abs() / tol).max()))


def _pad(lists, k, fill=-1):
    return _i32(*[x + [fill] * (k - len(x)) for row in lists for x in row]).view(len(lists), len(lists[0]), k)


def _random_lists(c, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in c.lens:
        nb = -(-n // c.bs)
        out.append([sorted(torch.randperm(nb, generator=g)[:int(torch.randint(1, k + 1, (1,), generator=g))].tolist())
                    for _ in range(c.KV)])
    return out


@pytest.mark.parametrize("dtype,D,H,KV,bs", [
    ("bf16", 128, 8, 2, 16), ("bf16", 64, 3, 1, 8), ("bf16", 256, 16, 1, 12), ("bf16", 64, 4, 4, 5),
    ("bf16", 128, 10, 2, 100), ("bf16", 256, 8, 8, 64), ("i8", 128, 8, 4, 4), ("i8", 256, 6, 2, 8),
    ("i8", 128, 4, 1, 64), ("bf16", 128, 128, 1, 16)])
def test_selected(kvc, dtype, D, H, KV, bs):
    lens = [1, 5 * bs, 11 * bs + 3, 30 * bs - 1]
    c = Built(kvc, "paged", dtype, lens, H, KV, D, bs=bs, seed=3)
    lists = _random_lists(c, 9)
    lists[3][0] = sorted(set(lists[3][0]) | {29})                # the partly filled last block
    ws = kvc.alloc_select_workspace(c.d, 10)
    first = None
    for _ in range(2):
        out = kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, _pad(lists, 10), ws, c.table)
        assert first is None or torch.equal(first, out)
        first = out
    _check_out(c, out, lists)
    assert kvc.get_error(ws) == 0


def test_selected_lists_with_gaps_and_absent_blocks(kvc):
    """Negative entries between others, blocks unmapped, not resident or past the position, empty lists."""
    lens = [300, 200, 250]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 128)
    c.table[0, 4] = -1
    dead = int(c.table[0, 9])
    mask = torch.ones(c.d.num_blocks, dtype=torch.bool)
    mask[dead] = False
    bits = kvc.pack_valid_bits(mask).cuda()
    entries = [[[-1, 2, 4, -5, 9, 11, -1, 18], [-1] * 8], [[0, 1, 2, 3, 4, 5, 12, 13], [12, -1, -1, -1, -1, -1, -1, 13]],
               [[-1] * 7 + [15], [15, 16] + [-1] * 6]]
    lists = [[[2, 11, 18], []], [[0, 1, 2, 3, 4, 5, 12], [12]], [[15], [15]]]
    ws = kvc.alloc_select_workspace(c.d, 8)
    out = kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, _i32(*sum(sum(entries, []), [])).view(3, 2, 8),
                                        ws, c.table, valid_bits=bits)
    _check_out(c, out, lists)
    assert kvc.get_error(ws) == 0


def test_selected_reports_bad_entries(kvc):
    lens = [300, 200]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 128)
    ws = kvc.alloc_select_workspace(c.d, 5)

    def run(entries, lists):
        out = kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, _i32(*sum(sum(entries, []), [])).view(2, 2, 5),
                                            ws, c.table)
        _check_out(c, out, lists)
        return kvc.get_error(ws)

    good = [[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]]
    ok = [[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]]
    # twice the same, descending, past the table, a wild value
    assert run([[[1, 1, 2, 5, 5], [7, 3, 8, 8, 9]], good], [[[1, 2, 5], [7, 8, 9]], ok]) == kvc.KVC_DEV_BAD_ENTRY
    far = c.table.shape[1]
    assert run([[[1, far, 2, 2 ** 31 - 1, 5], good[1]], good], [[[1, 2, 5], ok[1]], ok]) == kvc.KVC_DEV_BAD_ENTRY
    assert run([good, good], [ok, ok]) == 0
    c.table[0, 2] = c.d.num_blocks + 7
    assert run([good, good], [[[0, 1, 3, 4], ok[1]], ok]) == kvc.KVC_DEV_BAD_BLOCK


@pytest.mark.parametrize("dtype", ["bf16", "i8"])
@pytest.mark.parametrize("ns", [0, 1, 7, 200])
def test_selected_long_lists_and_splits(kvc, dtype, ns):
    lens = [16 * 700, 16 * 3 + 1, 16 * 400 + 5]
    c = Built(kvc, "paged", dtype, lens, 4, 2, 128, num_splits=ns)
    k = 520
    lists = _random_lists(c, 500, seed=ns)
    lists[0][0] = list(range(0, 700, 2))
    ws = kvc.alloc_select_workspace(c.d, k)
    out = kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, _pad(lists, k), ws, c.table)
    _check_out(c, out, lists)
    assert kvc.get_error(ws) == 0


def test_selected_one_sequence_and_many(kvc):
    c = Built(kvc, "paged", "bf16", [5000], 8, 8, 64)
    lists = _random_lists(c, 200)
    ws = kvc.alloc_select_workspace(c.d, 200)
    _check_out(c, kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, _pad(lists, 200), ws, c.table), lists)
    n = 150
    c = Built(kvc, "paged", "bf16", [33 + (i * 13) % 50 for i in range(n)], 4, 1, 64, bs=8)
    lists = _random_lists(c, 4)
    ws = kvc.alloc_select_workspace(c.d, 4)
    _check_out(c, kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, _pad(lists, 4), ws, c.table), lists)


def test_selected_baked_rope(kvc):
    lens = [150, 131]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 64, rope="baked", qstd=1.0)
    lists = [[[0, 3, 9], [1, 2]], [[8], [0, 4, 5, 8]]]
    ws = kvc.alloc_select_workspace(c.d, 4)
    out = kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, _pad(lists, 4), ws, c.table)
    turned = plain.rotate(c.q.double(), c.pos.double(), plain.frequencies(64)[0], 1.0, "half")
    # the rotated query is rounded to bf16: scores off by 2^-8 sum |q_i k_i| scale, twice in a weight
    qk = max(float(torch.einsum("hd,lhd->hl", turned[b].abs(), c.rows(b, range(n))[0].abs().repeat_interleave(4, 1)).amax())
             for b, n in enumerate(lens)) * c.scale
    _check_out(c, out, lists, q=turned, rel=REL + math.expm1(2 * 2.0 ** -8 * qk))


def test_selected_idle_sequences(kvc):
    lens = [150, 131, 90]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 64)
    lists = [[[0, 3, 9], [1, 2]], [[8], [0, 4]], [[0], [5]]]
    ws = kvc.alloc_select_workspace(c.d, 3)
    out = kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, _i32(149, -1, 89), _pad(lists, 3), ws, c.table)
    assert kvc.get_error(ws) == kvc.KVC_DEV_BAD_POSITION
    assert not out[1].any()
    _check_out(c, out, lists, skip=(1,))


def test_offsets_past_32_bits(kvc):
    """Blocks, codes and steps behind 2^32 elements of the cache and 2^31 bytes of the bounds."""
    KV, D, bs, nblocks = 8, 128, 16, 1100000
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=2, q_heads=8, kv_heads=KV, head_dim=D, block_size=bs,
                      num_blocks=nblocks, max_blocks_per_seq=8)
    cache, bounds = kvc.alloc_cache(d), kvc.alloc_bounds(d)
    assert bounds.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    table = _i32(nblocks - 1, 5, 700000, nblocks - 9, 1, 2, 3, 4, nblocks - 2, 9, 800000, 10, 11, 12, 13, 14).view(2, 8)
    for blk in table.flatten().tolist():
        cache[0, :, blk] = torch.randn(2, KV, bs, D, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(2, 8, D, generator=g, device="cuda").to(torch.bfloat16)
    pos, ws = _i32(127, 120), kvc.alloc_select_workspace(d, 4)
    kvc.block_bounds(d, cache, 0, bounds, _i32(0, 0), 128, ws, table, n_tok=_i32(128, 121))
    got = kvc.select_blocks(d, bounds, 0, q, pos, 4, ws, table)
    out = kvc.decode_attention_selected(d, cache, 0, q, pos, got, ws, table)
    codes, steps = kvc.bounds_views(d, bounds)
    for b in range(2):
        at = table[b].long()
        want = part.select(codes[0][at].cpu(), steps[0][at].cpu(), q[b].cpu(), list(range(8)), 8, 4, 1, 1, 1)
        assert got[b].tolist() == want
        for h in range(KV):
            k, v = (cache[0, i, at[want[h]], h].reshape(-1, D)[:64 if b == 0 else 57].double() for i in (0, 1))
            o, w = part.attend(q[b, h:h + 1].double(), k, v, D ** -0.5)
            mass = w @ v.abs()
            assert ((out[b, h].double() - o[0]).abs() <= REL * mass[0] + 2.0 ** -8 * (o[0].abs() + REL * mass[0]) + 1e-6).all()
    assert kvc.get_error(ws) == 0


def test_long_cache_step_and_graph(kvc):
    """As a server uses it: prepare, append, bounds, select, attend, captured in one graph and replayed while the
    positions advance; with k over all blocks it equals plain decode attention, and small k matches the lists."""
    B, H, KV, D, bs, k = 3, 8, 2, 64, 16, 40
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=B, q_heads=H, kv_heads=KV, head_dim=D, block_size=bs,
                      num_blocks=100, max_blocks_per_seq=20)
    cache, state = kvc.alloc_cache(d, fill=float("nan")), kvc.BlockState(d)
    ws, other, bounds = kvc.alloc_select_workspace(d, k), kvc.alloc_workspace(d), kvc.alloc_bounds(d)
    pos = _i32(0, 0, 0)
    q = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    kn, vn = (torch.empty(B, KV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    blocks, few = torch.empty(B, KV, k, dtype=torch.int32, device="cuda"), torch.empty(B, KV, 3, dtype=torch.int32, device="cuda")
    out, part_out = torch.empty_like(q), torch.empty_like(q)

    def step():
        kvc.block_prepare(d, cache, pos, state, ws)
        kvc.append(d, cache, 0, kn, vn, pos, ws, block_table=state.table)
        kvc.block_bounds(d, cache, 0, bounds, pos, 1, ws, state.table)
        kvc.select_blocks(d, bounds, 0, q, pos, k, ws, state.table, valid_bits=state.valid_bits, blocks=blocks)
        kvc.decode_attention_selected(d, cache, 0, q, pos, blocks, ws, state.table, valid_bits=state.valid_bits, out=out)
        kvc.select_blocks(d, bounds, 0, q, pos, 3, ws, state.table, valid_bits=state.valid_bits, blocks=few)
        kvc.decode_attention_selected(d, cache, 0, q, pos, few, ws, state.table, valid_bits=state.valid_bits, out=part_out)

    def renew():
        for x in (q, kn, vn):
            x.copy_(torch.randn(x.shape, device="cuda"))

    renew()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(1, 150):
        pos.add_(1)
        renew()
        graph.replay()
        if t % 30 == 1 or t == 149:
            ref = kvc.decode_attention(d, cache, 0, q, pos, other, block_table=state.table, valid_bits=state.valid_bits)
            assert float((ref.float() - out.float()).abs().max()) < 6e-2
            nb = t // bs + 1
            assert blocks[1, 1].tolist() == list(range(nb)) + [-1] * (k - nb)
            codes, steps = kvc.bounds_views(d, bounds)
            for b in range(B):
                at = state.table[b, :nb].long()
                want = part.select(codes[0][at].cpu(), steps[0][at].cpu(), q[b].cpu(), list(range(nb)), nb, 3, 1, 1, H // KV)
                assert [[x for x in r if x >= 0] for r in few[b].tolist()] == want
                for h in range(KV):
                    kk, vv = (cache[0, i, at[want[h]], h].reshape(-1, D).double() for i in (0, 1))
                    n = len(want[h]) * bs - (nb * bs - 1 - t)
                    o, w = part.attend(q[b, h * 4:h * 4 + 4].double(), kk[:n], vv[:n], D ** -0.5)
                    mass = w @ vv[:n].abs()
                    err = (part_out[b, h * 4:h * 4 + 4].double() - o).abs()
                    assert (err <= REL * mass + 2.0 ** -8 * (o.abs() + REL * mass) + 1e-6).all()
    assert kvc.get_error(ws) == 0


def test_calls_at_once_on_two_streams(kvc):
    runs = []
    for seed, lens in ((1, [900, 700, 655, 40]), (2, [2100, 2060])):
        c = Built(kvc, "paged", "bf16", lens, 8, 2, 128, seed=seed)
        bounds = _bounds(kvc, c, [0] * len(lens), lens)
        ws = kvc.alloc_select_workspace(c.d, 12)
        blocks = kvc.select_blocks(c.d, bounds, c.layer, c.q, c.pos, 12, ws, c.table)
        out = kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, blocks, ws, c.table)
        runs.append((c, bounds, ws, blocks, out, torch.empty_like(blocks), torch.empty_like(out), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, bounds, ws, _, _, blocks, out, s in runs:
            kvc.select_blocks(c.d, bounds, c.layer, c.q, c.pos, 12, ws, c.table, blocks=blocks, stream=s)
            kvc.decode_attention_selected(c.d, c.cache, c.layer, c.q, c.pos, blocks, ws, c.table, out=out, stream=s)
    torch.cuda.synchronize()
    for c, _, ws, want_b, want, blocks, out, _ in runs:
        assert torch.equal(blocks, want_b) and torch.equal(out, want)
        assert kvc.get_error(ws) == 0
