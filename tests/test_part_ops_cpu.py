"""Refusals and sizes of the operators on caches read or kept in part, and of the path append: checked on the
host before anything is launched (no GPU)."""

import ctypes

import pytest
import torch

A = 1 << 20          # a 16-byte aligned address that nothing reads
PAGED = dict(layout="paged", rope="none", dtype="bf16", layers=2, batch=3, q_heads=8, kv_heads=2, head_dim=128,
             block_size=16, num_blocks=12, max_blocks_per_seq=4)
RING = dict(layout="ring", rope="none", dtype="bf16", layers=2, batch=3, q_heads=8, kv_heads=2, head_dim=128, window=100)


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _all(call, kvc, null, align16, align4=()):
    for name in null:
        assert call(**{name: None}) == kvc.KVC_ERR_NULL, name
    for name in align16:
        assert call(**{name: A + 8}) == kvc.KVC_ERR_ALIGN, name
    for name in align4:
        assert call(**{name: A + 2}) == kvc.KVC_ERR_ALIGN, name
    assert call(layer=2) == kvc.KVC_ERR_ARG and call(layer=-1) == kvc.KVC_ERR_ARG


def test_bounds_refusals(kvc):
    L = kvc.lib()

    def call(base=PAGED, cache=A, layer=0, bounds=A, pos=A, n=4, table=A, ws=A, short=0, **kw):
        d = kvc.make_desc(**dict(base, **kw))
        return L.kvc_block_bounds(ctypes.byref(d), cache, layer, bounds, pos, n, None, table, ws,
                                  kvc.workspace_bytes(d) - short, None)

    _all(call, kvc, ("cache", "bounds", "pos", "table", "ws"), ("cache", "bounds", "ws"))
    assert call(n=0) == kvc.KVC_ERR_ARG and call(short=1) == kvc.KVC_ERR_WORKSPACE
    assert call(base=RING) == kvc.KVC_ERR_DESC and call(head_dim=96) == kvc.KVC_ERR_UNSUPPORTED
    d = kvc.make_desc(**PAGED)
    assert kvc.bounds_bytes(d) == 2 * 12 * 2 * (2 * 128 + 4)
    assert kvc.bounds_bytes(kvc.make_desc(**RING)) == 0
    with pytest.raises(kvc.KvcError):
        kvc.alloc_bounds(kvc.make_desc(**RING))
    buf = torch.arange(kvc.bounds_bytes(d), dtype=torch.int64).to(torch.uint8)
    codes, steps = kvc.bounds_views(d, buf)
    assert codes.shape == (2, 12, 2, 2, 128) and steps.shape == (2, 12, 2)
    assert codes.data_ptr() == buf.data_ptr() and steps.data_ptr() == buf.data_ptr() + codes.numel()


def test_select_refusals(kvc):
    L = kvc.lib()

    def call(base=PAGED, layer=0, bounds=A, q=A, pos=A, k=4, first=1, recent=1, table=A, blocks=A, ws=A, short=0, **kw):
        d = kvc.make_desc(**dict(base, **kw))
        n = kvc.select_workspace_bytes(d, k) - short if short else 1 << 40
        return L.kvc_select_blocks(ctypes.byref(d), bounds, layer, q, pos, k, first, recent, table, None, blocks, ws, n,
                                   None)

    _all(call, kvc, ("bounds", "q", "pos", "table", "blocks", "ws"), ("bounds", "q", "ws"), ("blocks",))
    for kw in (dict(k=0), dict(k=-1), dict(k=(1 << 24) + 1), dict(first=-1), dict(recent=0), dict(first=2, recent=3),
               dict(first=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert call(**kw) == kvc.KVC_ERR_ARG, kw
    assert call(base=RING) == kvc.KVC_ERR_DESC and call(short=1) == kvc.KVC_ERR_WORKSPACE
    assert call(q_heads=258) == kvc.KVC_ERR_UNSUPPORTED
    d = kvc.make_desc(**PAGED)
    assert kvc.select_workspace_bytes(d, 4) > kvc.workspace_bytes(d)
    assert kvc.select_workspace_bytes(d, 0) == 0 and kvc.select_workspace_bytes(kvc.make_desc(**RING), 4) == 0
    with pytest.raises(kvc.KvcError):
        kvc.alloc_select_workspace(d, 0)


def test_selected_refusals(kvc):
    L = kvc.lib()

    def call(base=PAGED, cache=A, layer=0, q=A, pos=A, blocks=A, k=4, table=A, out=A, ws=A, short=0, **kw):
        d = kvc.make_desc(**dict(base, **kw))
        n = kvc.select_workspace_bytes(d, k) - short if short else 1 << 40
        return L.kvc_decode_attention_selected(ctypes.byref(d), cache, layer, q, pos, blocks, k, table, None, out, ws, n,
                                               None)

    _all(call, kvc, ("cache", "q", "pos", "blocks", "table", "out", "ws"), ("cache", "q", "out", "ws"), ("blocks",))
    assert call(k=0) == kvc.KVC_ERR_ARG and call(short=1) == kvc.KVC_ERR_WORKSPACE
    assert call(dtype="f32") == kvc.KVC_ERR_UNSUPPORTED and call(q_heads=258) == kvc.KVC_ERR_UNSUPPORTED
    assert call(base=RING) == kvc.KVC_ERR_DESC
    # rows of a list are counted in 32 bits
    assert call(k=1 << 20, block_size=4096, num_blocks=2) == kvc.KVC_ERR_ARG


def test_weighed_refusals(kvc):
    L = kvc.lib()

    def call(base=PAGED, cache=A, layer=0, q=A, pos=A, table=A, decay=1.0, weights=A, out=A, ws=A, short=0, **kw):
        d = kvc.make_desc(**dict(base, **kw))
        n = kvc.weighed_workspace_bytes(d) - short if short else 1 << 40
        return L.kvc_decode_attention_weighed(ctypes.byref(d), cache, layer, q, pos, table, None, decay, weights, out, ws,
                                              n, None)

    _all(call, kvc, ("cache", "q", "pos", "table", "weights", "out", "ws"), ("cache", "q", "out", "ws"), ("weights",))
    for decay in (-0.1, 1.5, float("nan"), float("inf")):
        assert call(decay=decay) == kvc.KVC_ERR_ARG
    assert call(short=1) == kvc.KVC_ERR_WORKSPACE and call(dtype="f32") == kvc.KVC_ERR_UNSUPPORTED
    assert call(base=RING) == kvc.KVC_ERR_DESC
    d = kvc.make_desc(**PAGED)
    assert kvc.weighed_workspace_bytes(d) >= kvc.workspace_bytes(d) + 3 * 8 * 64 * 4
    assert kvc.weighed_workspace_bytes(kvc.make_desc(**dict(PAGED, dtype="f32"))) == 0
    with pytest.raises(kvc.KvcError):
        kvc.alloc_weighed_workspace(kvc.make_desc(**RING))


def test_evict_refusals(kvc):
    L = kvc.lib()

    def call(base=PAGED, weights=A, pos=A, keep=3, first=1, recent=1, table=A, ref=A, stack=A, count=A, ws=A, short=0, **kw):
        d = kvc.make_desc(**dict(base, **kw))
        return L.kvc_block_evict(ctypes.byref(d), weights, pos, keep, first, recent, table, None, ref, stack, count, ws,
                                 kvc.workspace_bytes(d) - short, None)

    for name in ("weights", "pos", "table", "ref", "stack", "count", "ws"):
        assert call(**{name: None}) == kvc.KVC_ERR_NULL, name
    assert call(ws=A + 8) == kvc.KVC_ERR_ALIGN and call(weights=A + 2) == kvc.KVC_ERR_ALIGN
    assert call(short=1) == kvc.KVC_ERR_WORKSPACE
    for kw in (dict(first=-1), dict(recent=0), dict(keep=1), dict(first=2, recent=2), dict(keep=-5)):
        assert call(**kw) == kvc.KVC_ERR_ARG, kw
    assert call(base=RING) == kvc.KVC_ERR_DESC


def test_path_refusals(kvc):
    L = kvc.lib()

    def call(base=PAGED, cache=A, layer=0, k=A, v=A, T=8, pos=A, path=A, P=4, n=A, table=A, ws=A, short=0, **kw):
        d = kvc.make_desc(**dict(base, **kw))
        return L.kvc_append_path(ctypes.byref(d), cache, layer, k, v, T, pos, path, P, n, table, ws,
                                 kvc.workspace_bytes(d) - short, None)

    _all(call, kvc, ("cache", "k", "v", "pos", "path", "table", "ws"), ("cache", "k", "v", "ws"), ("path", "n"))
    assert call(T=0) == kvc.KVC_ERR_ARG and call(P=0) == kvc.KVC_ERR_ARG and call(short=1) == kvc.KVC_ERR_WORKSPACE
    assert call(head_dim=96) == kvc.KVC_ERR_UNSUPPORTED


def test_binding_checks(kvc):
    """Shapes, types and devices are checked before the library is called (CPU tensors are refused)."""
    d = kvc.make_desc(**PAGED)
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(3, 4, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    kv = torch.zeros(3, 5, 2, 128, dtype=torch.bfloat16)
    cache = torch.zeros(kvc.cache_shape(d), dtype=torch.bfloat16)
    bounds = torch.zeros(kvc.bounds_bytes(d), dtype=torch.uint8)
    w = torch.zeros(3, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.block_bounds(d, cache, 0, bounds, i, 1, ws, table)
    with pytest.raises(ValueError, match="bounds holds"):
        kvc._take_bounds(kvc._sizes_of(d), bounds[:100], 0)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.select_blocks(d, bounds, 0, q, i, 4, ws, table)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.decode_attention_selected(d, cache, 0, q, i, torch.zeros(3, 2, 4, dtype=torch.int32), ws, table)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.decode_attention_weighed(d, cache, 0, q, i, w, ws, table)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.append_path(d, cache, 0, kv, kv, i, torch.zeros(3, 2, dtype=torch.int32), i, ws, table)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.block_evict(d, kvc.BlockState(d, device="cpu"), w, i, 3, ws)


def test_tree_refusals(kvc):
    L = kvc.lib()

    def call(base=PAGED, cache=A, layer=0, q=A, k=A, v=A, T=8, pos=A, parent=A, table=A, out=A, ws=A, short=0, **kw):
        d = kvc.make_desc(**dict(base, **kw))
        n = kvc.tree_workspace_bytes(d, T) - short if short else 1 << 40
        return L.kvc_tree_attention(ctypes.byref(d), cache, layer, q, k, v, T, pos, parent, table, None, out, ws, n, None)

    _all(call, kvc, ("cache", "q", "k", "v", "pos", "parent", "table", "out", "ws"), ("cache", "q", "k", "v", "out", "ws"),
         ("parent",))
    assert call(T=0) == kvc.KVC_ERR_ARG and call(T=kvc.KVC_TREE_MAX + 1) == kvc.KVC_ERR_ARG
    assert call(short=1) == kvc.KVC_ERR_WORKSPACE
    for kw in (dict(dtype="f32"), dict(dtype="i8"), dict(block_size=12), dict(block_size=48), dict(block_size=100),
               dict(q_heads=258), dict(base=RING, rope="read_time"), dict(base=RING, window=7), dict(head_dim=96)):
        assert call(**kw) == kvc.KVC_ERR_UNSUPPORTED, kw
        kw = dict(kw)
        assert kvc.tree_workspace_bytes(kvc.make_desc(**dict(kw.pop("base", PAGED), **kw)), 8) == 0
    d = kvc.make_desc(**PAGED)
    assert kvc.tree_workspace_bytes(d, 8) > kvc.workspace_bytes(d)
    with pytest.raises(kvc.KvcError):
        kvc.alloc_tree_workspace(d, 65)
    q = torch.zeros(3, 5, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(3, 5, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.tree_attention(d, kv, 0, q, kv, kv, torch.zeros(3, dtype=torch.int32), torch.zeros(3, 5, dtype=torch.int32),
                           torch.zeros(64, dtype=torch.uint8))


def test_longest_tables(kvc):
    """Tables of more than 2^30 blocks a sequence are refused by every call that walks them: their indices are 32
    bits, a whole CTA's stride past the end."""
    L = kvc.lib()

    def calls(maxb):
        d = kvc.make_desc(**dict(PAGED, batch=1, block_size=1, max_blocks_per_seq=maxb))
        r = ctypes.byref(d)
        return (L.kvc_block_bounds(r, A, 0, A, A, 4, None, A, A, 0, None),
                L.kvc_select_blocks(r, A, 0, A, A, 4, 1, 1, A, None, A, A, 0, None),
                L.kvc_decode_attention_selected(r, A, 0, A, A, A, 4, A, None, A, A, 0, None),
                L.kvc_decode_attention_weighed(r, A, 0, A, A, A, None, 1.0, A, A, A, 0, None),
                L.kvc_block_evict(r, A, A, 3, 1, 1, A, None, A, A, A, A, 0, None)), (
            kvc.bounds_bytes(d) > 0, kvc.select_workspace_bytes(d, 4) > 0, kvc.weighed_workspace_bytes(d) > 0)

    assert calls((1 << 30) + 1) == ((kvc.KVC_ERR_UNSUPPORTED,) * 5, (False,) * 3)
    assert calls(1 << 30) == ((kvc.KVC_ERR_WORKSPACE,) * 5, (True,) * 3)
