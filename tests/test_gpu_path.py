"""kvc_append_path on the GPU: the rows of the path where kvc_append would put them, nothing else touched."""

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


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _desc(kvc, layout, dtype, B, KV, D, rope="none", window=12, sinks=3, bs=8):
    paged = layout == "paged"
    return kvc.make_desc(layout, rope, dtype, layers=2, batch=B, q_heads=KV, kv_heads=KV, head_dim=D,
                         window=0 if paged else window, sinks=sinks if layout == "sink_ring" else 0,
                         block_size=bs if paged else 0, num_blocks=40 if paged else 0,
                         max_blocks_per_seq=8 if paged else 0)


def _setup(kvc, d, T, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    act = kvc.desc_dtype(d)
    k, v = (torch.randn(d.batch, T, d.kv_heads, d.head_dim, generator=g, device="cuda").to(act) for _ in range(2))
    cache = kvc.alloc_cache(d)
    cache.view(torch.uint8).copy_(torch.randint(0, 100, cache.view(torch.uint8).shape, generator=g, device="cuda"))
    table = None
    if d.layout == 2:
        table = torch.randperm(40, generator=torch.Generator().manual_seed(seed))[:d.batch * 8].view(d.batch, 8)
        table = table.to(torch.int32).cuda()
    return k, v, cache, table, kvc.alloc_workspace(d)


CASES = [("ring", "bf16", 64), ("ring", "i8", 128), ("sink_ring", "f32", 64), ("sink_ring", "bf16", 256),
         ("paged", "f32", 128), ("paged", "bf16", 128), ("paged", "i8", 256), ("paged", "f32", 256), ("paged", "bf16", 64)]


@pytest.mark.parametrize("layout,dtype,D", CASES)
@pytest.mark.parametrize("rope", ["none", "baked"])
def test_equals_append_of_the_gathered_rows(kvc, layout, dtype, D, rope):
    """One sequence at a time, kvc_append of the path's rows puts the same values to the same places."""
    B, T, P, KV = 4, 20, 16, 4
    d = _desc(kvc, layout, dtype, B, KV, D, rope)
    k, v, cache, table, ws = _setup(kvc, d, T)
    g = torch.Generator().manual_seed(1)
    path = torch.stack([torch.randperm(T, generator=g)[:P].sort().values for _ in range(B)]).to(torch.int32).cuda()
    path[0, 3] = path[0, 2]                                 # one token twice
    n, pos = [16, 1, 0, 7], [0, 30, 5, 41]
    want = cache.clone()
    for b in range(B):
        if n[b]:
            one = torch.full((B,), -10 ** 6, dtype=torch.int32)     # the others: positions that append nothing
            one[b] = pos[b]
            at = path[:, :n[b]].long()
            rows = torch.arange(B, device="cuda")[:, None]
            kvc.append(d, want, 1, k[rows, at].contiguous(), v[rows, at].contiguous(), one.cuda(), ws, block_table=table)
    kvc.append_path(d, cache, 1, k, v, _i32(*pos), path, _i32(*n), ws, block_table=table)
    assert kvc.get_error(ws) == 0
    if rope == "none" or dtype == "i8":
        assert torch.equal(cache.view(torch.uint8), want.view(torch.uint8))
        return
    # the same angles and products; another order of their sum moves a value by half a step at most, twice
    step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -22
    same = cache.view(torch.uint8) == want.view(torch.uint8)
    assert float(same.float().mean()) > 0.99
    a, b = cache.double(), want.double()
    moved = a != b
    assert ((a - b).abs()[moved] <= step * b.abs()[moved] + 1e-6).all()


def test_rotation_against_float64(kvc):
    d = _desc(kvc, "paged", "f32", 2, 2, 64, "baked")
    k, v, cache, table, ws = _setup(kvc, d, 5)
    kvc.append_path(d, cache, 0, k, v, _i32(9, 50), _i32(0, 2, 4, 1, 3, 4).view(2, 3), None, ws, block_table=table)
    for b, (p0, toks) in enumerate(((9, (0, 2, 4)), (50, (1, 3, 4)))):
        for j, t in enumerate(toks):
            p = p0 + j
            at = int(table[b, p // 8])
            want = plain.rotate(k[b, t].double(), torch.tensor(p, device="cuda"), plain.frequencies(64)[0], 1.0, "half")
            # (an angle is off by 2e-7 at most, its sine and cosine by as much again; products and sum 2^-23)
            assert ((cache[0, 0, at, :, p % 8].double() - want).abs() <= 1e-6 * k[b, t].double().abs().amax(-1, keepdim=True)).all()
            assert torch.equal(cache[0, 1, at, :, p % 8], v[b, t])


def test_long_paths_over_a_small_window(kvc):
    """A row that a later one of the same call overwrites is not written."""
    for layout in ("ring", "sink_ring"):
        d = _desc(kvc, layout, "bf16", 1, 2, 64, window=4)
        k, v, cache, _, ws = _setup(kvc, d, 30)
        path = _i32(*range(30)).view(1, 30)
        kvc.append_path(d, cache, 1, k, v, _i32(0), path, None, ws)
        S = d.sinks
        for p in list(range(S)) + list(range(26, 30)):
            slot = p if p < S else S + (p - S) % 4
            assert torch.equal(cache[1, 0, 0, :, slot], k[0, p]) and torch.equal(cache[1, 1, 0, :, slot], v[0, p])


def test_bad_entries(kvc):
    d = _desc(kvc, "paged", "bf16", 3, 2, 64)
    k, v, cache, table, ws = _setup(kvc, d, 4)
    before = cache.clone()

    def run(pos, path, n):
        cache.copy_(before)
        kvc.append_path(d, cache, 0, k, v, _i32(*pos), _i32(*path).view(3, 2), _i32(*n), ws, block_table=table)
        return kvc.get_error(ws)

    def rows(b, *ps):
        return [cache[0, 0, int(table[b, p // 8]), :, p % 8] for p in ps]

    # indices out of range in the counted part alone; their position stays as it was
    assert run([0, 8, 16], [1, 4, -1, 2, 3, 99], [2, 2, 1]) == kvc.KVC_DEV_BAD_ENTRY
    assert torch.equal(rows(0, 0)[0], k[0, 1]) and torch.equal(rows(1, 9)[0], k[1, 2]) and torch.equal(rows(2, 16)[0], k[2, 3])
    for b, p in ((0, 1), (1, 8), (2, 17)):
        assert torch.equal(rows(b, p)[0], before[0, 0, int(table[b, p // 8]), :, p % 8])
    assert run([0, 8, 16], [0, 1, 0, 1, 0, 1], [3, -2, 2]) == kvc.KVC_DEV_BAD_ENTRY
    assert torch.equal(rows(0, 1)[0], k[0, 1])
    assert run([0, -1, -5], [0, 1, 0, 1, 0, 1], [1, 2, 2]) == 0
    assert run([63, 0, 0], [0, 1, 0, 1, 0, 1], [2, 0, 0]) == kvc.KVC_DEV_BAD_POSITION
    assert run([2 ** 31 - 1, 0, 0], [0, 1, 0, 1, 0, 1], [2, 0, 0]) == kvc.KVC_DEV_BAD_POSITION
    table[0, 1] = -1
    assert run([7, 0, 0], [0, 1, 0, 1, 0, 1], [2, 0, 0]) == kvc.KVC_DEV_UNMAPPED_APPEND
    table[0, 1] = 40
    assert run([7, 0, 0], [0, 1, 0, 1, 0, 1], [2, 0, 0]) == kvc.KVC_DEV_BAD_BLOCK
