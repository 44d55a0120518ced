"""A NaN in a query is the answer of its row: weights of NaN scores are NaN, so every value of that
(token, q head) row is, and no other row changes by a bit.  A row that attends nothing stays zero,
and NaN keys that a row does not attend do not reach it.

Capped scores share a reciprocal among four keys, so that what a row does not attend may move the rounding
of its own scores: v = 1 / (e^(2 x / cap) + 1) by a few 2^-23 of itself, a capped score by 2^-20 cap, a
weight by twice that in numerator and denominator (1e-3 for caps to 200), and the output by one step more."""

import pytest
import torch

from tests.cache_builder import Built

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _slopes(H):
    return (2.0 ** (-6.0 * torch.arange(1, H + 1, device="cuda") / H)).float()


def _nan_rows(run, q, rows):
    """run(q) with a NaN in one value of each of `rows` (indices of q's leading dimensions): these rows are NaN
    throughout, the others as without it."""
    want = run(q)
    assert torch.isfinite(want.float()).all()
    bad = q.clone()
    for j, r in enumerate(rows):
        bad[r][(37 * j + 5) % q.shape[-1]] = NAN
    got = run(bad)
    for r in rows:
        assert got[r].isnan().all(), (r, got[r])
        got[r] = want[r]
    assert torch.equal(got, want)


MODS = [dict(), dict(softcap=20.0), dict(softcap=200.0), dict(slopes=True), dict(softcap=5.0, slopes=True)]


def _score(kvc, H, mods, start=None):
    return kvc.make_score(mods.get("softcap", 0.0), _slopes(H) if mods.get("slopes") else None, start)


def _prefill(kvc, c, T, score, q, k, v):
    """prefill_scored on a copy of the cache."""
    ws = kvc.alloc_prefill_workspace(c.d, T)
    pos0 = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    out = kvc.prefill_scored(c.d, c.cache.clone(), c.layer, q, k, v, pos0, ws, score, block_table=c.table)
    assert kvc.get_error(ws) == 0
    return out


def _chunk(c, T, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(c.lens)
    q = (torch.randn(B, T, c.H, c.D, generator=g, device="cuda") * 2).to(c.act)
    k, v = (torch.randn(B, T, c.KV, c.D, generator=g, device="cuda").to(c.act) for _ in range(2))
    return q, k, v


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("i8", 128)])
@pytest.mark.parametrize("layout,kw", [("paged", dict(lens=(0, 500, 64))), ("ring", dict(lens=(0, 300, 900), window=256)),
                                       ("sink_ring", dict(lens=(2, 300, 900), window=252, sinks=4))])
def test_nan_query_of_a_scored_prefill(kvc, mods, dtype, D, layout, kw):
    T = 70
    c = Built(kvc, layout, dtype, H=8, KV=2, D=D, new=T, **kw)
    q, k, v = _chunk(c, T)
    rows = [(0, 0, 0), (0, 69, 7), (1, 0, 3), (1, 33, 0), (2, 64, 5), (2, 65, 4)]
    _nan_rows(lambda x: _prefill(kvc, c, T, _score(kvc, 8, mods), x, k, v), q, rows)


@pytest.mark.parametrize("mods", MODS)
def test_nan_query_and_keys_outside_the_document(kvc, mods):
    """Tokens that attend nothing give zeros whatever their query holds; NaN keys behind a token, or of another
    document in the same tile, do not reach it."""
    T, H = 130, 4
    c = Built(kvc, "paged", "bf16", (0, 77), H, 1, 128, new=T)
    q, k, v = _chunk(c, T)
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    pos0 = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    start = (pos0[:, None] + (t // 40 * 40)[None]).contiguous()       # documents of 40 tokens
    start[:, 5::7] = 10000                                            # and tokens of none
    score = _score(kvc, H, mods, start)
    want = _prefill(kvc, c, T, score, q, k, v)
    assert not want[:, 5::7].any()
    bad = q.clone()
    bad[:, 5::7] = NAN
    assert torch.equal(_prefill(kvc, c, T, score, bad, k, v), want)
    keys = k.clone()
    keys[0, 39], keys[0, 129], keys[1, 80] = NAN, NAN, NAN
    got = _prefill(kvc, c, T, score, q, keys, v)
    touched = torch.zeros(2, T, dtype=torch.bool, device="cuda")
    touched[0, 39], touched[0, 129], touched[1, 80:120] = True, True, True
    touched[:, 5::7] = False
    move = (got.float() - want.float()).abs()
    assert (move <= 1e-3 * v.abs().max() + 2.0 ** -7 * want.float().abs())[~touched].all()
    if not mods.get("softcap"):
        assert torch.equal(got[~touched], want[~touched])
    assert got[touched].isnan().all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,prefix", [((200, 190, 210, 130), 128), ((300, 257, 256, 256), 256)])
def test_nan_query_of_a_shared_decode(kvc, D, lens, prefix):
    """Groups of two; a sequence whose keys are all shared, and one alone."""
    bs, tables, at = 16, [], prefix // 16
    for n in lens:
        own = -(-n // bs) - at
        tables.append(list(range(at)) + [at + sum(len(t) - at for t in tables) + i for i in range(own)])
    c = Built(kvc, "paged", "bf16", lens, 8, 2, D, bs=bs, tables=tables)
    ws = kvc.alloc_shared_workspace(c.d)
    group = torch.tensor([1, 1, 1, -1], dtype=torch.int32, device="cuda")
    _nan_rows(lambda x: kvc.decode_attention_shared(c.d, c.cache, c.layer, x, c.pos, group, ws, c.table), c.q,
              [(0, 0), (1, 5), (2, 7), (3, 2)])
    assert kvc.get_error(ws) == 0


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("layout,kw", [("ring", dict(lens=(1, 50, 1200), window=64)),
                                       ("ring", dict(lens=(1, 50, 9000), window=4096)),
                                       ("paged", dict(lens=(1, 40, 1200), bs=16)), ("paged", dict(lens=(700,), bs=16))])
def test_nan_query_of_a_decode(kvc, dtype, layout, kw, plain):
    """One part and many, for the plain call as well."""
    c = Built(kvc, layout, dtype, H=4, KV=2, D=128, **kw)
    B = len(c.lens)
    rows = [(b, (b + 1) % 4) for b in range(B)]
    if plain:
        _nan_rows(lambda x: kvc.decode_attention(c.d, c.cache, c.layer, x, c.pos, c.ws, block_table=c.table), c.q, rows)
    else:
        for mods in MODS:
            start = torch.zeros(B, dtype=torch.int32, device="cuda")
            score = _score(kvc, 4, mods, start)
            run = lambda x: kvc.decode_attention_scored(c.d, c.cache, c.layer, x, c.pos, c.ws, score, block_table=c.table)
            _nan_rows(run, c.q, rows)
            start.fill_(2 ** 30)                  # nothing attended: zeros, whatever the query holds
            assert not run(torch.full_like(c.q, NAN)).any()
    assert kvc.get_error(c.ws) == 0
