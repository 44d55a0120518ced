"""kvc_append_qk on the GPU against its formula in float64: q_out, the rows written, and the rows
left as they were.

Tolerance of a value y of a row x: the operator rounds once (half a step of y) after fp32
arithmetic.  The angle is off by at most two fp32 roundings of a number up to pi (3.8e-7) and
sincosf by 2^-22; the products and their sum add three roundings: under 1e-6 (|x'_a| + |x'_b|)
together.  The norm's factor (a sum of at most 256 squares over a butterfly: 13 roundings, rsqrtf:
2 ulp, two products) is within 1.2e-6 relative.  4e-6 max|x'| mag covers both."""

import math

import pytest
import torch

from tests import plain_ops as plain

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.bfloat16}


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _table(B, maxb, blocks, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(blocks, generator=g)[:B * maxb].view(B, maxb).to(torch.int32)


def _run(kvc, layout="paged", dtype="bf16", B=3, H=8, KV=2, D=128, n_new=1, pos=(0, 5, 100), n_tok=None, window=0,
         sinks=0, bs=16, maxb=24, layers=2, layer=1, rot=128, pairs="half", scaling="none", norm=True, offset=0.0,
         eps=1e-6, packed=True, inplace=False, rope="none", stream=None, seed=0, sides="qk"):
    act = ACT[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = kvc.make_desc(layout, rope, dtype, layers=layers, batch=B, q_heads=H, kv_heads=KV, head_dim=D, window=window,
                      sinks=sinks, block_size=bs if layout == "paged" else 0,
                      num_blocks=B * maxb + 4 if layout == "paged" else 0,
                      max_blocks_per_seq=maxb if layout == "paged" else 0)
    cache = kvc.alloc_cache(d, fill=3.0)
    ws = kvc.alloc_workspace(d)
    table = _table(B, maxb, d.num_blocks, seed).cuda() if layout == "paged" else None
    x = torch.randn(B, n_new, (H + 2 * KV) * D, generator=g, device="cuda").to(act)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in x.split([H * D, KV * D, KV * D], -1))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(act) if norm and "q" in sides else None
    kw = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(act) if norm and "k" in sides else None
    spec = dict(dim=rot, scaling=scaling, factor=4.0 if scaling != "none" else 1.0,
                original_len=2048 if scaling in ("yarn", "bands") else 0, fast=4.0 if scaling == "bands" else 32.0)
    qk = kvc.make_qk(d, rotary=kvc.make_rotary(pairs, **spec) if rot else None, q_weight=qw, k_weight=kw, eps=eps,
                     weight_offset=offset)
    pos_t = torch.tensor(pos, dtype=torch.int32, device="cuda")
    n_t = None if n_tok is None else torch.tensor(n_tok, dtype=torch.int32, device="cuda")
    q_out = q if inplace else torch.full((B, n_new, H, D), 7.0, dtype=act, device="cuda")
    q64, k64, v64 = q.double(), k.double(), v.double()
    before = cache.clone()
    kvc.append_qk(d, cache, layer, q, k, v, pos_t, ws, qk, n_tok=n_t, block_table=table, q_out=q_out, stream=stream)
    torch.cuda.synchronize()
    # the formula
    freq, mag = plain.frequencies(**spec) if rot else ([], 1.0)
    P = pos_t.cpu().long()[:, None] + torch.arange(n_new)
    yq = plain.norm(q64, qw, eps, offset)
    yk = plain.norm(k64, kw, eps, offset)
    mq, mk = yq.abs().amax(-1, keepdim=True), yk.abs().amax(-1, keepdim=True)
    yq, yk = plain.rotate(yq, P.cuda(), freq, mag, pairs), plain.rotate(yk, P.cuda(), freq, mag, pairs)
    half = plain.HALF_STEP[act]
    real = torch.zeros(B, n_new, dtype=torch.bool)
    for b in range(B):
        n = n_new if n_tok is None else min(n_tok[b], n_new)
        real[b, :max(n, 0)] = True
    real &= P >= 0
    # q_out
    want = torch.where(real[..., None, None].cuda(), yq, q64 if inplace else torch.full_like(yq, 7.0))
    tol = half * want.abs() + 4e-6 * mq * mag * (1 + half)
    bad = (q_out.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float((q_out.double() - want).abs().max()))
    # the cache
    if dtype == "i8":
        codes, scales = (t.clone() for t in kvc.int8_views(d, cache))
        c0, s0 = kvc.int8_views(d, before)
    else:
        codes, c0 = cache.clone(), before
    tc = table.cpu() if table is not None else None
    for b in range(B):
        rows = {}
        for i in range(n_new):
            p = int(P[b, i])
            if not real[b, i]:
                continue
            if layout == "paged":
                lb = p // bs
                if lb < maxb:
                    rows[(int(tc[b, lb]), p % bs)] = i
            else:
                rows[(b, plain.slot_of(layout, p, window, sinks))] = i
        for (blk, r), i in rows.items():
            for which, y, m in ((0, yk, mk * mag), (1, v64, None)):
                ref = y[b, i]
                slack = 0.0 if m is None else 4e-6 * m[b, i]
                if dtype == "i8":
                    sc = scales[layer, which, blk, :, r].double()[:, None]
                    got = codes[layer, which, blk, :, r].double() * sc
                    top = ref.abs().amax(-1, keepdim=True) / 127
                    assert ((sc - top).abs() <= 1e-6 * top + slack / 127).all()
                    # half a code step, the quotient's rounding, and the value's own error
                    assert ((got - ref).abs() <= 0.5 * sc * (1 + 1e-4) + 127 * (sc - top).abs() + slack).all()
                    codes[layer, which, blk, :, r] = c0[layer, which, blk, :, r]
                    scales[layer, which, blk, :, r] = s0[layer, which, blk, :, r]
                else:
                    got = codes[layer, which, blk, :, r].double()
                    lim = (half * ref.abs() + slack * (1 + half)) if m is not None else torch.zeros_like(ref)
                    assert ((got - ref).abs() <= lim).all(), (b, i, which)
                    codes[layer, which, blk, :, r] = c0[layer, which, blk, :, r]
    assert torch.equal(codes, c0), "a row of no token was written"
    if dtype == "i8":
        assert torch.equal(scales, s0)
    return kvc.get_error(ws)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 128),
                                     ("f32", 256), ("i8", 128), ("i8", 256)])
@pytest.mark.parametrize("layout,kw", [
    ("paged", dict(pos=(0, 5, 100), bs=16)),
    ("paged", dict(pos=(0, 5, 100), bs=7, maxb=40)),
    ("ring", dict(window=40, pos=(0, 39, 1000), maxb=1)),
    ("sink_ring", dict(window=36, sinks=4, pos=(0, 3, 987600), maxb=1)),
])
@pytest.mark.parametrize("n_new", [1, 19])
def test_layouts_types_and_heads(kvc, dtype, D, layout, kw, n_new):
    kw = dict(kw)
    if dtype == "i8" and kw.get("bs") == 7:
        kw["KV"] = 4
        kw["H"] = 8
    assert _run(kvc, layout=layout, dtype=dtype, D=D, rot=D, n_new=n_new, **kw) == 0


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [0, 2, 16, 32, 50, 62, 64, 126, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
def test_rotated_parts(kvc, pairs, rot, dtype):
    assert _run(kvc, rot=rot, pairs=pairs, dtype=dtype, n_new=5, pos=(0, 90, 300)) == 0


@pytest.mark.parametrize("scaling", ["linear", "yarn", "bands"])
@pytest.mark.parametrize("rot,D", [(64, 64), (96, 128), (256, 256)])
def test_scaled_positions(kvc, scaling, rot, D):
    assert _run(kvc, scaling=scaling, rot=rot, D=D, layout="ring", window=64, maxb=1, n_new=9, dtype="f32",
                pos=(1, 4000, 1 << 20)) == 0


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 1), (24, 8), (64, 1), (7, 7)])
def test_head_counts(kvc, H, KV):
    assert _run(kvc, H=H, KV=KV, n_new=3) == 0


@pytest.mark.parametrize("norm,sides,offset", [(False, "qk", 0.0), (True, "q", 0.0), (True, "k", 0.0),
                                               (True, "qk", 1.0)])
def test_norm_choices(kvc, norm, sides, offset):
    assert _run(kvc, norm=norm, sides=sides, offset=offset, n_new=4) == 0


def test_padding_and_counts(kvc):
    """Left padding (negative positions), ragged counts, none at all, and counts past the call's."""
    assert _run(kvc, B=5, n_new=12, pos=(-3, 0, 7, -20, 40), n_tok=(12, 0, 5, 12, 99)) == 0
    # the last real token decides what a ring keeps, not the padding behind it
    assert _run(kvc, layout="ring", window=6, maxb=1, B=4, n_new=15, pos=(0, 100, 3, -2), n_tok=(15, 9, -1, 10)) == 0
    assert _run(kvc, layout="sink_ring", window=5, sinks=3, maxb=1, B=4, n_new=15, pos=(0, 100, 1, -2),
                n_tok=(15, 9, 2, 10)) == 0


def test_dense_and_in_place(kvc):
    assert _run(kvc, packed=False, n_new=6) == 0
    assert _run(kvc, packed=False, inplace=True, n_new=6) == 0
    assert _run(kvc, packed=False, inplace=True, n_new=1, rot=50) == 0


def test_positions_near_the_end_of_the_range(kvc):
    assert _run(kvc, layout="ring", window=50, maxb=1, n_new=4, dtype="f32",
                pos=(2 ** 31 - 1 - 4, 2 ** 31 - 5, 1 << 30)) == 0


def test_read_time_cache_takes_the_norms_alone(kvc):
    assert _run(kvc, layout="sink_ring", window=36, sinks=4, maxb=1, rot=0, rope="read_time", n_new=3) == 0


def test_bad_blocks_are_reported_and_skipped(kvc):
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=4, q_heads=4, kv_heads=2, head_dim=64, block_size=8,
                      num_blocks=6, max_blocks_per_seq=2)
    cache = kvc.alloc_cache(d, fill=1.0)
    ws = kvc.alloc_workspace(d)
    q, k, v = (torch.ones(4, n, 64, dtype=torch.bfloat16, device="cuda") for n in (4, 2, 2))
    table = torch.tensor([[0, -1], [6, 1], [2, 3], [4, 5]], dtype=torch.int32, device="cuda")
    qk = kvc.make_qk(d)
    for pos, bits in (((9, 3, 0, 0), kvc.KVC_DEV_UNMAPPED_APPEND | kvc.KVC_DEV_BAD_BLOCK),
                      ((0, 12, 16, -5), kvc.KVC_DEV_BAD_POSITION)):
        q_out = torch.zeros_like(q)
        kvc.append_qk(d, cache, 0, q, k, v, torch.tensor(pos, dtype=torch.int32, device="cuda"), ws, qk,
                      block_table=table, q_out=q_out)
        assert kvc.get_error(ws) == bits
        assert torch.equal(q_out[:3], q[:3])
    assert bool((q_out[3] == 0).all())


def test_offsets_past_32_bits(kvc):
    """A cache whose V half begins past 2^31 elements and ends past 2^32."""
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=2, q_heads=8, kv_heads=8, head_dim=128, block_size=16,
                      num_blocks=140000, max_blocks_per_seq=3)
    cache = kvc.alloc_cache(d)
    assert cache.numel() > 2 ** 32 and cache.numel() // 2 > 2 ** 31
    ws = kvc.alloc_workspace(d)
    table = torch.tensor([[139999, 0, 70000], [139998, 1, 5]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(2, 40, 8, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    kvc.append_qk(d, cache, 0, q, k, v, torch.zeros(2, dtype=torch.int32, device="cuda"), ws, kvc.make_qk(d),
                  block_table=table)
    for b in range(2):
        for i in (0, 15, 16, 33, 39):
            blk = int(table[b, i // 16])
            assert torch.equal(cache[0, 0, blk, :, i % 16], k[b, i])
            assert torch.equal(cache[0, 1, blk, :, i % 16], v[b, i])
    assert kvc.get_error(ws) == 0


def test_special_values_stay_in_their_rows(kvc):
    """An infinity or NaN outside the rotated part changes no other value; a zero row stays zero."""
    d = kvc.make_desc("ring", "none", "f32", layers=1, batch=1, q_heads=2, kv_heads=1, head_dim=128, window=8)
    cache, ws = kvc.alloc_cache(d, fill=0.0), kvc.alloc_workspace(d)
    q = torch.randn(1, 2, 128, device="cuda")
    q[0, 0, 100], q[0, 0, 101] = math.inf, math.nan
    k, v = torch.zeros(1, 1, 128, device="cuda"), torch.randn(1, 1, 128, device="cuda")
    v[0, 0, 3] = -math.inf
    pos = torch.tensor([3], dtype=torch.int32, device="cuda")
    w = torch.ones(128, device="cuda")
    for rot in (64, 36):
        out = kvc.append_qk(d, cache, 0, q, k, v, pos, ws, kvc.make_qk(d, kvc.make_rotary("half", dim=rot), k_weight=w))
        assert out[0, 0, 100] == math.inf and out[0, 0, 101].isnan()
        assert int(out.isfinite().sum()) == 254
        assert torch.equal(cache[0, 0, 0, 0, 3], torch.zeros(128, device="cuda"))
        assert torch.equal(cache[0, 1, 0, 0, 3], v[0, 0])


def test_graph_and_another_stream(kvc):
    """Captured into a graph and replayed on changed inputs; issued on a stream of its own."""
    side = torch.cuda.Stream()
    assert _run(kvc, n_new=3, stream=side, seed=3) == 0
    d = kvc.make_desc("ring", "none", "bf16", layers=1, batch=2, q_heads=4, kv_heads=2, head_dim=64, window=16)
    cache, ws = kvc.alloc_cache(d, fill=0.0), kvc.alloc_workspace(d)
    q, k, v = (torch.randn(2, n, 64, device="cuda").to(torch.bfloat16) for n in (4, 2, 2))
    pos = torch.tensor([0, 7], dtype=torch.int32, device="cuda")
    qk = kvc.make_qk(d, kvc.make_rotary("half", dim=64))
    out = torch.empty_like(q)
    kvc.append_qk(d, cache, 0, q, k, v, pos, ws, qk, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.append_qk(d, cache, 0, q, k, v, pos, ws, qk, q_out=out)
    for step in range(3):
        q.copy_(torch.randn_like(q.float()))
        k.copy_(torch.randn_like(k.float()))
        pos.add_(5)
        graph.replay()
        got, rows = out.clone(), cache.clone()
        want_cache = cache.clone()
        want = kvc.append_qk(d, want_cache, 0, q, k, v, pos, ws, qk)
        assert torch.equal(got, want) and torch.equal(rows, want_cache)
    assert kvc.get_error(ws) == 0
