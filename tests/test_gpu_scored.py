"""kvc_decode_attention_scored and kvc_prefill_scored on the GPU against the formula in float64.

Tolerances, for an output sum w_i v_i (weights w, scores s, fp32 statistics):
 - the fp32 kernel: a score is a sum of products in at most 13 dependent roundings of
   sum |q_i k_i| scale (under 60 for these inputs), a capped one is off by 6 2^-23 cap more; twice
   that is the relative error of a weight: under 2e-4 together, sums of weights included;
 - bf16 and INT8 decode: the same, at most 2^-24 D 60 (1e-3 for twice that), and each weight is
   rounded to bf16 (2^-8; fp16 2^-11 for INT8) before it meets v, and the output to bf16;
 - prefill: a weight's base-2 argument is rounded to fp16: off by half a step, 2^-7 below 32 (larger
   ones weigh under 2^-32), which changes the weight by ln 2 2^-7, in numerator and denominator, and
   the fp16 result by 2^-11 more, twice: 1.3e-2 together with what decode has;
 - a baked query is rounded to bf16 after its rotation: scores off by 2^-8 sum |q_i k_i| scale."""

import math

import pytest
import torch

from tests import plain_ops as plain
from tests.cache_builder import Built

pytestmark = pytest.mark.gpu

REL = {"f32": 2e-4, "bf16": 2.0 ** -8 + 1e-3, "i8": 2.0 ** -8 + 1e-3}


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


def _within(got, want, weight, rel, act):
    """|got - want| <= rel sum w |v| + half a step of the value."""
    tol = rel * weight + plain.HALF_STEP[act] * (want.abs() + rel * weight) + 1e-6
    bad = (got.double() - want).abs() > tol
    assert torch.isfinite(got.float()).all()
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


def _decode(kvc, layout, dtype, lens, H=8, KV=2, D=128, cap=0.0, bias=False, start=None, dead=(), poison=True, more=0.0,
            **kw):
    c = Built(kvc, layout, dtype, lens, H, KV, D, **kw)
    slopes = _slopes(H) if bias else None
    st = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    valid = None
    gone = set()
    if layout == "paged" and dead:
        mask = torch.ones(c.d.num_blocks, dtype=torch.bool)
        mask[list(dead)] = False
        valid = kvc.pack_valid_bits(mask).cuda()
        gone = set(dead)
    out = torch.full_like(c.q, float("nan"))
    if poison and start is not None:
        for b, n in enumerate(lens):
            c.poison(b, [p for p in c.kv[b] if p < max(0, start[b])])
    score = kvc.make_score(softcap=cap, slopes=slopes, start=st)
    for _ in range(2):            # the second call finds the workspace as the first left it
        out.fill_(float("nan"))
        kvc.decode_attention_scored(c.d, c.cache, c.layer, c.q, c.pos, c.ws, score, block_table=c.table,
                                    valid_bits=valid, out=out)
    assert kvc.get_error(c.ws) == 0
    for b, n in enumerate(lens):
        ps = plain.attended(layout, n - 1, c.window, c.sinks, max(0, start[b]) if start is not None else 0)
        ps = [p for p in ps if layout != "paged" or int(c.table[b, p // c.bs]) not in gone]
        if not ps:
            assert not out[b].any()
            continue
        k, v = c.rows(b, ps)
        dist = torch.tensor([[n - 1 - p for p in ps]], device="cuda")
        want, w = plain.attend(c.q[b].double()[None], k, v, dist, torch.ones_like(dist, dtype=torch.bool), c.scale,
                               cap, slopes)
        weight = torch.einsum("htl,lhd->thd", w, v.abs().repeat_interleave(H // KV, 1))
        _within(out[b], want[0], weight[0], REL[dtype] + more, c.act)
    return c, out


MODS = [dict(), dict(cap=20.0), dict(bias=True), dict(cap=5.0, bias=True)]


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 128),
                                     ("f32", 256), ("i8", 128), ("i8", 256)])
@pytest.mark.parametrize("layout,kw", [
    ("paged", dict(lens=(1, 77, 300), bs=16)),
    ("paged", dict(lens=(5, 130, 257), bs=64)),
    ("ring", dict(lens=(1, 99, 100, 1234), window=100)),
    ("sink_ring", dict(lens=(2, 60, 100, 1234), window=96, sinks=4)),
])
def test_decode_layouts_types_modifiers(kvc, mods, dtype, D, layout, kw):
    _decode(kvc, layout, dtype, D=D, **kw, **mods)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("layout,kw", [
    # starts: none, mid block, on a block, the token itself, past it (nothing attended), below 0
    ("paged", dict(lens=(200, 200, 200, 200, 200, 200), bs=16, start=(0, 37, 64, 199, 200, -7))),
    ("paged", dict(lens=(150, 3, 90), bs=24, start=(149, 3, 23))),
    ("ring", dict(lens=(500, 500, 500, 500, 40), window=100, start=(0, 450, 499, 500, 20))),
    ("sink_ring", dict(lens=(500, 500, 500, 500, 500, 40), window=96, sinks=4, start=(0, 2, 450, 499, 500, 3))),
])
def test_decode_starts(kvc, dtype, layout, kw):
    _decode(kvc, layout, dtype, cap=8.0, bias=True, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
def test_one_paged_sequence(kvc, dtype):
    """Planned inside the attention kernel without a start, by the planning kernel with one."""
    _decode(kvc, "paged", dtype, lens=(700,), bias=True)
    _decode(kvc, "paged", dtype, lens=(700,), bias=True, start=(333,))
    _decode(kvc, "paged", dtype, lens=(1,), cap=3.0)


@pytest.mark.parametrize("dtype", ["bf16", "i8"])
@pytest.mark.parametrize("bs", [8, 16, 20, 32, 128])
def test_paged_block_sizes_and_absent_blocks(kvc, dtype, bs):
    c, _ = _decode(kvc, "paged", dtype, lens=(1, 333, 190), bs=bs, bias=True, cap=10.0)
    dead = [int(c.table[1, 0]), int(c.table[1, 1]), int(c.table[2, 0]), int(c.table[0, 0])]
    _decode(kvc, "paged", dtype, lens=(1, 333, 190), bs=bs, bias=True, cap=10.0, dead=dead)
    _decode(kvc, "paged", dtype, lens=(1, 333, 190), bs=bs, bias=True, dead=dead, start=(0, 2 * bs + 1, 3))


@pytest.mark.parametrize("H,KV", [(1, 1), (2, 2), (6, 2), (12, 2), (24, 3), (16, 1), (5, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_groups(kvc, H, KV, dtype):
    _decode(kvc, "paged", dtype, lens=(90, 33), H=H, KV=KV, cap=12.0, bias=True, start=(7, 0))


@pytest.mark.parametrize("num_splits", [1, 2, 7, 64])
@pytest.mark.parametrize("layout,kw", [("ring", dict(window=512)), ("paged", dict(bs=16))])
def test_split_counts(kvc, num_splits, layout, kw):
    for dtype in ("bf16", "f32"):
        _decode(kvc, layout, dtype, lens=(1000, 3, 513), num_splits=num_splits, bias=True, start=(700, 0, 100), **kw)


def test_many_sequences(kvc):
    """More than the 64 sequences whose rows a CTA keeps in registers; some attend nothing."""
    lens = [(i * 37) % 150 + 1 for i in range(70)]
    start = [0 if i % 3 else lens[i] - (i % 5) for i in range(70)]
    _decode(kvc, "paged", "bf16", lens=lens, H=4, KV=1, cap=15.0, bias=True, start=start)
    _decode(kvc, "ring", "bf16", lens=lens, H=4, KV=1, window=64, cap=15.0, bias=True, start=start)
    _decode(kvc, "paged", "bf16", lens=(30, 40), start=(30, 40), bias=True)      # nothing at all


def test_far_positions_and_flat_slopes(kvc):
    """Distances from a position near 10^6, and the sinks' distance there."""
    _decode(kvc, "sink_ring", "f32", lens=(987654,), window=60, sinks=4, H=4, KV=1, D=64, bias=True)
    _decode(kvc, "sink_ring", "bf16", lens=(987654, 1 << 20), window=60, sinks=4, bias=True, cap=9.0)


def test_no_modifier_equals_plain_decode(kvc):
    """With no modifier set the result is decode attention's, to the rounding of its scaled query
    (which the scored form leaves unscaled)."""
    c, out = _decode(kvc, "paged", "bf16", lens=(100, 260))
    ref = kvc.decode_attention(c.d, c.cache, c.layer, c.q, c.pos, c.ws, block_table=c.table)
    assert float((ref.float() - out.float()).abs().max()) < 6e-2


def test_custom_scale_and_baked_rope(kvc):
    _decode(kvc, "paged", "bf16", lens=(50, 60), softmax_scale=0.25, cap=4.0)
    # baked: q rotated at its position inside the call; the cached keys are taken as they are
    lens, H, KV, D = (37, 80), 4, 2, 64
    c = Built(kvc, "paged", "bf16", lens, H, KV, D, rope="baked")
    out = kvc.decode_attention_scored(c.d, c.cache, c.layer, c.q, c.pos, c.ws, kvc.make_score(softcap=6.0),
                                      block_table=c.table)
    freq, _ = plain.frequencies(D)
    for b, n in enumerate(lens):
        k, v = c.rows(b, range(n))
        q = plain.rotate(c.q[b].double(), torch.tensor(n - 1, device="cuda"), freq, 1.0, "half")
        see = torch.ones(1, n, dtype=torch.bool, device="cuda")
        want, w = plain.attend(q[None], k, v, torch.zeros(1, n, device="cuda"), see, c.scale, 6.0)
        weight = torch.einsum("htl,lhd->thd", w, v.abs().repeat_interleave(H // KV, 1))
        qk = torch.einsum("hd,lhd->hl", q.abs(), k.abs().repeat_interleave(H // KV, 1)).amax() * c.scale
        _within(out[b], want[0], weight[0], REL["bf16"] + math.expm1(2 * 2.0 ** -8 * float(qk)), c.act)


def test_saturated_and_infinite_scores(kvc):
    """Scores far beyond the cap saturate at it; an infinite product counts as the cap."""
    for dtype in ("bf16", "f32"):
        c = Built(kvc, "ring", dtype, (9,), 2, 1, 64, window=16, qstd=200.0)
        c.q[0, 1, 0] = 3e38
        c.cache[c.layer, 0, 0, 0, 0, 0] = 3e38      # q . k overflows for head 1, key 0
        c.k[c.index[(0, 0)], 0, 0] = 3e38
        out = kvc.decode_attention_scored(c.d, c.cache, c.layer, c.q, c.pos, c.ws, kvc.make_score(softcap=2.0))
        k, v = c.rows(0, range(9))
        see = torch.ones(1, 9, dtype=torch.bool, device="cuda")
        want, w = plain.attend(c.q[0].double()[None], k, v, torch.zeros(1, 9, device="cuda"), see, c.scale, 2.0)
        _within(out[0], want[0], torch.einsum("htl,lhd->thd", w, v.abs().repeat_interleave(2, 1))[0], REL[dtype],
                c.act)


def _prefill(kvc, layout, dtype, lens, T, H=8, KV=2, D=128, cap=0.0, bias=False, docs=None, rope="none", seed=0, more=0.0,
             dead=lambda b, j: False, **kw):
    """lens[b]: tokens cached before the chunk (negative: the chunk starts with padding)."""
    have = [max(0, n) for n in lens]
    c = Built(kvc, layout, dtype, have, H, KV, D, rope=rope, seed=seed, new=T, **kw)
    B = len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (torch.randn(B, T, H, D, generator=g, device="cuda") * 2).to(c.act)
    k, v = (torch.randn(B, T, KV, D, generator=g, device="cuda").to(c.act) for _ in range(2))
    pos0 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    slopes = _slopes(H) if bias else None
    start = None
    if docs is not None:
        start = torch.tensor([[docs(b, i, lens[b]) for i in range(T)] for b in range(B)], dtype=torch.int32,
                             device="cuda")
        for b in range(B):
            low = int(start[b].min())
            c.poison(b, [p for p in c.kv[b] if p < low])
    ws = kvc.alloc_prefill_workspace(c.d, T)
    out = torch.full_like(q, float("nan"))
    ref_cache = c.cache.clone()
    valid = None
    if layout == "paged":      # dead(b, j): logical block j of sequence b, wholly cached, is not resident
        mask = torch.ones(c.d.num_blocks, dtype=torch.bool)
        for b in range(B):
            for j in range(have[b] // c.bs):
                if dead(b, j):
                    mask[int(c.table[b, j])] = False
        valid = kvc.pack_valid_bits(mask).cuda() if not mask.all() else None
    kvc.prefill_scored(c.d, c.cache, c.layer, q, k, v, pos0, ws, kvc.make_score(cap, slopes, start),
                       block_table=c.table, valid_bits=valid, out=out)
    assert kvc.get_error(ws) == 0
    kvc.append(c.d, ref_cache, c.layer, k, v, pos0, ws, block_table=c.table)
    assert torch.equal(c.cache.view(torch.uint8), ref_cache.view(torch.uint8))
    k64, v64 = k.double(), v.double()
    if dtype == "i8":     # the chunk's rows as the cache reads them back, bf16 of code * scale
        for x in (k64, v64):
            s = x.abs().amax(-1, keepdim=True).float() / 127
            code = (x.float() / s).round().clamp(-127, 127).double()       # the format's fp32 quotient
            x.copy_((code * s.double()).to(torch.bfloat16).double())
    for b in range(B):
        old = plain.attended(layout, have[b] - 1, c.window, c.sinks)
        if start is not None:
            old = [p for p in old if p >= int(start[b].min())]
        if layout == "paged":
            old = [p for p in old if (p // c.bs + 1) * c.bs > have[b] or not dead(b, p // c.bs)]
        kc, vc = c.rows(b, old) if old else (k64[b, :0], v64[b, :0])
        if dtype == "i8" and old:
            kc, vc = kc.to(torch.bfloat16).double(), vc.to(torch.bfloat16).double()
        first = min(T, max(0, -lens[b]))          # left padding, the whole chunk if need be
        t = torch.arange(lens[b] + first, lens[b] + T, device="cuda")
        p = torch.cat([torch.tensor(old, dtype=torch.long, device="cuda"), t])
        K, V = torch.cat([kc, k64[b, first:]]), torch.cat([vc, v64[b, first:]])
        see = p[None] <= t[:, None]
        if layout != "paged":
            see &= (p[None] < c.sinks) | (p[None] > t[:, None] - c.window)
        if start is not None:
            see &= p[None] >= start[b, first:].long()[:, None]
        want, w = plain.attend(q[b, first:].double(), K, V, t[:, None] - p[None], see, c.scale, cap, slopes)
        weight = torch.einsum("htl,lhd->thd", w, V.abs().repeat_interleave(H // KV, 1))
        assert not out[b, :first].any()
        _within(out[b, first:], want, weight, 2.0 ** -8 + 1.3e-2 + more, c.act)


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("i8", 128), ("i8", 256)])
@pytest.mark.parametrize("layout,kw", [
    ("paged", dict(lens=(0, 50, 333), bs=16)),
    ("ring", dict(lens=(0, 150, 1000), window=150)),
    ("sink_ring", dict(lens=(2, 150, 1000), window=150, sinks=4)),
])
def test_prefill_layouts_types_modifiers(kvc, mods, dtype, D, layout, kw):
    _prefill(kvc, layout, dtype, T=37, D=D, **kw, **mods)


@pytest.mark.parametrize("layout,kw", [("paged", dict(bs=8)), ("paged", dict(bs=64)), ("ring", dict(window=400)),
                                       ("sink_ring", dict(window=396, sinks=4))])
@pytest.mark.parametrize("name", ["packed", "short", "inside", "alone", "empty", "mixed"])
def test_prefill_documents(kvc, layout, kw, name):
    docs = {
        "packed": lambda b, i, n: max(n, 0) + (i // 90) * 90 if i >= 20 else n // 2,   # the first goes on from the cache
        "short": lambda b, i, n: max(0, n + (i // 3) * 3),                            # three tokens each
        "inside": lambda b, i, n: max(0, n - 5 - 7 * b),                              # one start inside the cache
        "alone": lambda b, i, n: max(0, n + i),                                       # each token itself
        "empty": lambda b, i, n: max(0, n + i) + (1 if i % 2 else 0),                 # every second token nothing
        "mixed": lambda b, i, n: (i * 131) % (max(n, 0) + i + 1),                     # no order at all
    }[name]
    _prefill(kvc, layout, "bf16", lens=(0, 77, 300), T=201, docs=docs, bias=True, cap=15.0, **kw)


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 128, 300])
def test_prefill_lengths(kvc, T):
    _prefill(kvc, "paged", "bf16", lens=(0, 63, 64), T=T, cap=10.0, bias=True, H=4, KV=1)


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 1), (6, 1), (7, 1), (10, 2), (48, 1)])
def test_prefill_head_groups(kvc, H, KV):
    """Groups that do not divide the 128 rows of a tile leave its last rows empty."""
    _prefill(kvc, "ring", "bf16", lens=(0, 90), T=70, H=H, KV=KV, window=128, cap=10.0, bias=True)


def test_prefill_left_padding(kvc):
    _prefill(kvc, "paged", "bf16", lens=(-9, 5, -70), T=66, bias=True, cap=10.0)
    _prefill(kvc, "paged", "bf16", lens=(-9, 5, -70), T=66, bias=True, docs=lambda b, i, n: max(0, n + i - 3))


def test_prefill_all_masked(kvc):
    """No token of the chunk attends anything: zeros, and the chunk is appended all the same."""
    _prefill(kvc, "paged", "bf16", lens=(0, 40), T=50, docs=lambda b, i, n: 100000, cap=5.0)


def test_one_step_then_prefill_in_a_graph(kvc):
    """Captured, then replayed on other inputs: equal to the direct call, twice."""
    c = Built(kvc, "paged", "bf16", (300, 40, 77), 8, 2, 128)
    start = torch.tensor([100, 0, 78], dtype=torch.int32, device="cuda")
    score = kvc.make_score(7.0, _slopes(8), start)
    out = torch.empty_like(c.q)
    call = lambda ws, o: kvc.decode_attention_scored(c.d, c.cache, c.layer, c.q, c.pos, ws, score,
                                                     block_table=c.table, out=o)
    call(c.ws, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c.ws, out)
    other = kvc.alloc_workspace(c.d)
    for step in range(3):
        c.q.copy_(torch.randn_like(c.q.float()))
        start[0] += 50
        graph.replay()
        assert torch.equal(out, call(other, torch.empty_like(out)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvc.decode_attention_scored(c.d, c.cache, c.layer, c.q, c.pos, c.ws, score, block_table=c.table, stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    assert kvc.get_error(c.ws) == 0


def test_norm_rotary_append_then_scored_attention(kvc):
    """The run of a layer: a prompt through kvc_append_qk and the scored prefill's attention of the
    same tokens, then single steps, against full attention over normed and rotated rows."""
    H, KV, D, bs, steps = 8, 2, 64, 16, 4
    lens = (45, 20)
    d = kvc.make_desc("paged", "none", "bf16", layers=1, batch=2, q_heads=H, kv_heads=KV, head_dim=D, block_size=bs,
                      num_blocks=8, max_blocks_per_seq=4)
    cache, ws = kvc.alloc_cache(d, fill=float("nan")), kvc.alloc_workspace(d)
    table = torch.tensor([[3, 1, 7, 0], [6, 2, 5, 4]], dtype=torch.int32, device="cuda")
    T = max(lens) + steps
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(2, T, n, D, generator=g, device="cuda").to(torch.bfloat16) for n in (H, KV, KV))
    w = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    rot = kvc.make_rotary("interleaved", dim=32, scaling="yarn", factor=2.0, original_len=64)
    qk = kvc.make_qk(d, rot, w, w)
    score = kvc.make_score(12.0, _slopes(H), torch.tensor([9, 0], dtype=torch.int32, device="cuda"))
    n_tok = torch.tensor(lens, dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    qr = torch.zeros(2, T, H, D, dtype=torch.bfloat16, device="cuda")
    kvc.append_qk(d, cache, 0, q, k, v, zero, ws, qk, n_tok=n_tok, block_table=table, q_out=qr)
    freq, mag = plain.frequencies(32, scaling="yarn", factor=2.0, original_len=64)
    P = torch.arange(T, device="cuda")[None].expand(2, T)
    yq, yk = (plain.rotate(plain.norm(x.double(), w, 1e-6, 0.0), P, freq, mag, "interleaved").to(torch.bfloat16)
              .double() for x in (q, k))
    for step in range(steps):
        at = [n + step for n in lens]
        pos = torch.tensor(at, dtype=torch.int32, device="cuda")
        take = lambda x: torch.stack([x[b, at[b]] for b in range(2)]).contiguous()
        qs = kvc.append_qk(d, cache, 0, take(q), take(k), take(v), pos, ws, qk, block_table=table)
        out = kvc.decode_attention_scored(d, cache, 0, qs, pos, ws, score, block_table=table)
        for b in range(2):
            t = at[b]
            p = torch.arange((9, 0)[b], t + 1, device="cuda")
            dist = (t - p)[None]
            want, wt = plain.attend(yq[b, t][None], yk[b, p], v[b, p].double(), dist,
                                    torch.ones_like(dist, dtype=torch.bool), D ** -0.5, 12.0, _slopes(H))
            weight = torch.einsum("htl,lhd->thd", wt, v[b, p].double().abs().repeat_interleave(H // KV, 1))
            # stored q and k may sit a step (2^-7) from the reference's own rounding at a tie's edge
            qk_sum = torch.einsum("hd,lhd->hl", yq[b, t].abs(), yk[b, p].abs().repeat_interleave(H // KV, 1)).amax()
            rel = REL["bf16"] + math.expm1(4 * 2.0 ** -7 * float(qk_sum) * D ** -0.5 * 0.02)
            _within(out[b], want[0], weight[0], rel, torch.bfloat16)
    assert kvc.get_error(ws) == 0


@pytest.mark.parametrize("cap", [2.0 ** -10, 1024.0])
def test_smallest_and_largest_caps(kvc, cap):
    more = 12 * 2.0 ** -23 * cap      # a capped score is off by 6 2^-23 cap, a weight by twice that
    for dtype in ("bf16", "f32"):
        _decode(kvc, "ring", dtype, lens=(70, 3), window=64, H=4, KV=2, D=64, cap=cap, more=more)
    _prefill(kvc, "paged", "bf16", lens=(0, 70), T=40, cap=cap, more=more)        # a fixed reference, and a sought one
    _prefill(kvc, "paged", "bf16", lens=(0, 70), T=40, cap=cap, bias=True, more=more)


@pytest.mark.parametrize("cap", [0.5, 30.0, 34.0, 35.0, 51.0, 53.0, 80.0])
@pytest.mark.parametrize("vmag", [1.0, 1e16, 1e-3])
def test_prefill_scores_at_the_cap(kvc, cap, vmag):
    """Scores at +cap and -cap: rows that see only the one, only the other, and both; large values."""
    T, H, D, dev = 150, 4, 64, "cuda"
    c = Built(kvc, "paged", "bf16", (0, 0, 0), H, 1, D, new=T)
    g = torch.Generator(device=dev).manual_seed(3)
    sign = torch.ones(3, T, device=dev)
    sign[0] = -1
    sign[2] = torch.where(torch.rand(T, generator=g, device=dev) < 0.5, 1.0, -1.0)
    q = torch.full((3, T, H, D), 1000.0, device=dev, dtype=torch.bfloat16)
    k = (sign[:, :, None, None] * torch.full((1, 1, 1, D), 1000.0, device=dev)).to(torch.bfloat16)
    v = (torch.randn(3, T, 1, D, generator=g, device=dev) * vmag).to(torch.bfloat16)
    pos0 = torch.zeros(3, dtype=torch.int32, device=dev)
    ws = kvc.alloc_prefill_workspace(c.d, T)
    out = kvc.prefill_scored(c.d, c.cache, c.layer, q, k, v, pos0, ws, kvc.make_score(cap), block_table=c.table)
    assert kvc.get_error(ws) == 0
    t = torch.arange(T, device=dev)
    for b in range(3):
        want, w = plain.attend(q[b].double(), k[b].double(), v[b].double(), t[:, None] - t[None], t[None] <= t[:, None],
                               c.scale, cap)
        weight = torch.einsum("htl,lhd->thd", w, v[b].double().abs().repeat_interleave(H, 1))
        _within(out[b].double() / vmag, want / vmag, weight / vmag, 2.0 ** -8 + 1.3e-2, c.act)


def test_starts_at_the_ends_of_the_range(kvc):
    """The smallest and largest int32 as starts: nothing masked, everything masked."""
    lo, hi = -2 ** 31, 2 ** 31 - 1
    for dtype in ("bf16", "f32", "i8"):
        _decode(kvc, "paged", dtype, lens=(90, 90, 90), start=(lo, hi, 5), bias=True)
        _decode(kvc, "ring", dtype, lens=(300, 300, 300), window=100, start=(lo, hi, 250), cap=5.0)
    _prefill(kvc, "paged", "bf16", lens=(0, -5, 70), T=66, docs=lambda b, i, n: (0, hi, lo, max(0, n + i))[i % 4])


def test_calls_at_once_on_two_streams(kvc):
    """Each with its own workspace: the results of the calls alone."""
    a = Built(kvc, "paged", "bf16", (900, 333, 64), 8, 2, 128, seed=1)
    b = Built(kvc, "ring", "bf16", (900, 333, 64), 8, 2, 128, window=512, seed=2)
    sa, sb = kvc.make_score(9.0, _slopes(8)), kvc.make_score(0.0, _slopes(8))
    ra = kvc.decode_attention_scored(a.d, a.cache, a.layer, a.q, a.pos, a.ws, sa, block_table=a.table)
    rb = kvc.decode_attention_scored(b.d, b.cache, b.layer, b.q, b.pos, b.ws, sb)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.empty_like(ra), torch.empty_like(rb)
    torch.cuda.synchronize()
    for _ in range(20):
        kvc.decode_attention_scored(a.d, a.cache, a.layer, a.q, a.pos, a.ws, sa, block_table=a.table, out=oa, stream=one)
        kvc.decode_attention_scored(b.d, b.cache, b.layer, b.q, b.pos, b.ws, sb, out=ob, stream=two)
    torch.cuda.synchronize()
    assert torch.equal(oa, ra) and torch.equal(ob, rb)
    assert kvc.get_error(a.ws) == 0 and kvc.get_error(b.ws) == 0


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("bf16", 64), ("i8", 16)])
@pytest.mark.parametrize("mods", [dict(cap=6.0), dict(bias=True), dict(cap=6.0, bias=True)])
def test_prefill_absent_blocks(kvc, dtype, bs, mods):
    """Cached blocks that are not resident, some, all but one, all."""
    _prefill(kvc, "paged", dtype, lens=(400, 333, 200), T=70, bs=bs,
             dead=lambda b, j: (j % 3 == 1, j != 2, True)[b], **mods)
    _prefill(kvc, "paged", dtype, lens=(400, 333, 200), T=70, bs=bs, dead=lambda b, j: j % 2 == b % 2,
             docs=lambda b, i, n: max(0, n - 150 + 3 * i), **mods)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (256, "bf16"), (256, "i8")])
def test_long_chunks_of_other_head_dims(kvc, D, dtype):
    """More tiles than stages before, inside and behind the chunk's diagonal."""
    for mods in (dict(cap=20.0), dict(bias=True)):
        _prefill(kvc, "paged", dtype, lens=(0, 900), T=520, D=D, H=4, KV=1, **mods)
        _prefill(kvc, "sink_ring", dtype, lens=(40, 2000), T=520, D=D, H=4, KV=1, window=600, sinks=4, **mods)
