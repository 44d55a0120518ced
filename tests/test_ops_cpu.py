"""Refusals and host arithmetic of the serving-step operators, without a GPU: every argument error
comes back before anything is issued (with no GPU, a launch would give KVC_ERR_CUDA)."""

import ctypes
import math
import re
import os

import pytest
import torch

from tests import plain_ops as plain

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20   # a fake, 16-byte aligned "device" address: never dereferenced on these paths


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _desc(kvc, **kw):
    base = dict(layout="ring", rope="none", dtype="bf16", layers=2, batch=3, q_heads=8, kv_heads=2, head_dim=128,
                window=100)
    base.update(kw)
    return kvc.make_desc(**base)


def _struct_fields(name):
    with open(os.path.join(ROOT, "include", "kvc.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    body = re.search(r"typedef struct %s \{([^}]*)\}" % name, src).group(1)
    return [ln.strip().rstrip(";") for ln in body.strip().splitlines() if ln.strip()]


def test_structs_match_the_header(kvc):
    width = {"int32_t": ctypes.c_int32, "float": ctypes.c_float}
    for name, cls in (("kvc_rotary", kvc.KvcRotary), ("kvc_qk", kvc.KvcQk), ("kvc_score", kvc.KvcScore)):
        fields = _struct_fields(name)
        assert len(fields) == len(cls._fields_), name
        for text, (field, t) in zip(fields, cls._fields_):
            ctype, ident = text.rsplit(" ", 1)
            assert ident.split("[")[0] == field, (name, text)
            if "*" in ctype:
                assert t is ctypes.c_void_p, (name, text)
            elif "[" in ident:
                assert t._length_ == int(ident.split("[")[1][:-1]) and t._type_ is ctypes.c_uint64
            else:
                assert t is width[ctype], (name, text)


@pytest.mark.parametrize("spec", [
    dict(dim=128), dict(dim=64, base=500000.0), dict(dim=50, scaling="linear", factor=8.0),
    dict(dim=128, scaling="yarn", factor=4.0, original_len=4096),
    dict(dim=64, scaling="yarn", factor=40.0, original_len=4096, base=10000.0, fast=16.0, slow=2.0),
    dict(dim=2, scaling="yarn", factor=2.0, original_len=128),
    dict(dim=128, scaling="bands", factor=8.0, original_len=8192, base=500000.0, fast=4.0, slow=1.0),
    dict(dim=256, scaling="linear", factor=0.01),           # over a turn for each position
])
def test_rotary_tables(kvc, spec):
    """turns / 2^64 is the fraction of a turn f_i / (2 pi), to float64 rounding (2^-52 of the frequency)."""
    r = kvc.make_rotary("half", **spec)
    # the parameters as the struct holds them, fp32
    freq, mag = plain.frequencies(**dict(spec, factor=r.factor, base=r.base))
    for i, f in enumerate(freq):
        turn = f / (2 * math.pi)
        got = r.turns[i] / 2.0 ** 64
        diff = abs(got - (turn - math.floor(turn)))
        assert min(diff, 1 - diff) <= 8 * 2.0 ** -52 * max(turn, 1e-3), i
    assert abs(r.magnitude - mag) <= 2.0 ** -23 * mag and r.ready == 1
    assert kvc.make_rotary("half", **dict(spec, magnitude=0.5)).magnitude == 0.5


@pytest.mark.parametrize("spec", [
    dict(dim=3), dict(dim=258), dict(dim=-2), dict(dim=64, base=1.0), dict(dim=64, base=float("nan")),
    dict(dim=64, scaling="linear", factor=0.0), dict(dim=64, scaling="linear", factor=float("inf")),
    dict(dim=64, scaling="yarn", factor=4.0), dict(dim=64, scaling="yarn", factor=4.0, original_len=100, fast=1.0),
    dict(dim=64, scaling="bands", factor=4.0, original_len=100, slow=0.0), dict(dim=64, magnitude=-1.0),
])
def test_rotary_refusals(kvc, spec):
    with pytest.raises(kvc.KvcError) as e:
        kvc.make_rotary("half", **spec)
    assert e.value.code == kvc.KVC_ERR_ARG
    assert kvc.lib().kvc_rotary_init(None) == kvc.KVC_ERR_NULL


def test_append_qk_refusals(kvc):
    L = kvc.lib()

    def call(d=None, cache=A, layer=0, q=A, k=A, v=A, qs=0, ks=0, vs=0, n=1, pos=A, table=None, qk="none", out=A,
             ws=A, ws_n=None, **kw):
        d = d if d is not None else _desc(kvc, **kw)
        if qk == "none":
            qk = kvc.KvcQk(None, None, None, 1e-6, 0.0)
        n_ws = kvc.workspace_bytes(d) if ws_n is None else ws_n
        return L.kvc_append_qk(ctypes.byref(d), cache, layer, q, k, v, qs, ks, vs, n, pos, None, table,
                               ctypes.byref(qk) if qk is not None else None, out, ws, n_ws, None)

    for name in ("cache", "q", "k", "v", "pos", "out", "ws", "qk"):
        assert call(**{name: None}) == kvc.KVC_ERR_NULL, name
    for name in ("cache", "q", "k", "v", "out", "ws"):
        assert call(**{name: A + 8}) == kvc.KVC_ERR_ALIGN, name
    assert call(qk=kvc.KvcQk(None, A + 2, None, 1e-6, 0.0)) == kvc.KVC_ERR_ALIGN
    assert call(qs=8 * 128 + 4) == kvc.KVC_ERR_ALIGN
    assert call(qs=8 * 128 - 8) == kvc.KVC_ERR_ARG
    assert call(ks=-8) == kvc.KVC_ERR_ARG
    assert call(layer=2) == kvc.KVC_ERR_ARG and call(layer=-1) == kvc.KVC_ERR_ARG
    assert call(n=0) == kvc.KVC_ERR_ARG
    assert call(qk=kvc.KvcQk(None, None, None, -1.0, 0.0)) == kvc.KVC_ERR_ARG
    assert call(qk=kvc.KvcQk(None, None, None, float("nan"), 0.0)) == kvc.KVC_ERR_ARG
    d = _desc(kvc)
    assert call(d=d, ws_n=kvc.workspace_bytes(d) - 1) == kvc.KVC_ERR_WORKSPACE
    assert call(head_dim=96) == kvc.KVC_ERR_UNSUPPORTED
    paged = dict(layout="paged", window=0, block_size=16, num_blocks=10, max_blocks_per_seq=4)
    assert call(**paged) == kvc.KVC_ERR_NULL                     # no block table
    # a cache that rotates by itself
    assert call(rope="baked") == kvc.KVC_ERR_UNSUPPORTED
    rot = kvc.make_rotary("half", dim=128)
    qk = kvc.KvcQk(ctypes.addressof(rot), None, None, 1e-6, 0.0)
    assert call(rope="read_time", qk=qk) == kvc.KVC_ERR_UNSUPPORTED
    # a rotary wider than the head, or never made ready
    assert call(head_dim=64, qk=qk) == kvc.KVC_ERR_ARG
    raw = kvc.KvcRotary(0, 64, 0, 0, 10000.0, 1.0, 32.0, 1.0, 1.0)
    assert call(qk=kvc.KvcQk(ctypes.addressof(raw), None, None, 1e-6, 0.0)) == kvc.KVC_ERR_ARG


def test_append_qk_binding_checks(kvc):
    """Shapes and types are checked before the library is called (CPU tensors are refused)."""
    d = _desc(kvc)
    qk = kvc.make_qk(d)
    x = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.append_qk(d, x, 0, x, x, x, x, x, qk)
    with pytest.raises(ValueError, match="n_new"):
        kvc.append_qk(d, x, 0, x[0], x, x, x, x, qk)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.make_qk(d, q_weight=torch.zeros(128, dtype=torch.bfloat16))


def test_scored_refusals(kvc):
    L = kvc.lib()
    none = kvc.KvcScore(None, None, 0.0)

    def decode(score=none, cache=A, q=A, pos=A, out=A, layer=0, table=None, **kw):
        d = _desc(kvc, **kw)
        return L.kvc_decode_attention_scored(ctypes.byref(d), cache, layer, q, pos, table, None,
                                             ctypes.byref(score) if score is not None else None, out, A,
                                             kvc.workspace_bytes(d), None)

    def prefill(score=none, T=16, table=None, n_ws=1 << 40, **kw):
        d = _desc(kvc, **kw)
        return L.kvc_prefill_scored(ctypes.byref(d), A, 0, A, A, A, T, A, table, None,
                                    ctypes.byref(score) if score is not None else None, A, A, n_ws, None)

    for call in (decode, prefill):
        assert call(score=None) == kvc.KVC_ERR_NULL
        for cap in (-1.0, float("nan"), float("inf"), 1e-4, 2000.0):
            assert call(score=kvc.KvcScore(None, None, cap)) == kvc.KVC_ERR_ARG
        assert call(score=kvc.KvcScore(A + 2, None, 0.0)) == kvc.KVC_ERR_ALIGN
        assert call(score=kvc.KvcScore(None, A + 1, 0.0)) == kvc.KVC_ERR_ALIGN
        assert call(rope="read_time") == kvc.KVC_ERR_UNSUPPORTED
    assert decode(q=None) == kvc.KVC_ERR_NULL and decode(out=A + 4) == kvc.KVC_ERR_ALIGN
    assert decode(layer=2) == kvc.KVC_ERR_ARG
    paged = dict(layout="paged", window=0, block_size=16, num_blocks=10, max_blocks_per_seq=4)
    assert decode(**paged) == kvc.KVC_ERR_NULL and prefill(**paged) == kvc.KVC_ERR_NULL
    assert prefill(dtype="f32") == kvc.KVC_ERR_UNSUPPORTED
    assert prefill(T=101) == kvc.KVC_ERR_UNSUPPORTED                       # longer than the window
    assert prefill(q_heads=258) == kvc.KVC_ERR_UNSUPPORTED                 # a group of 129 heads
    assert prefill(**dict(paged, block_size=12), table=A) == kvc.KVC_ERR_UNSUPPORTED
    assert prefill(T=0) == kvc.KVC_ERR_ARG and prefill(n_ws=64) == kvc.KVC_ERR_WORKSPACE


def test_shared_refusals(kvc):
    L = kvc.lib()
    base = dict(layout="paged", window=0, block_size=16, num_blocks=10, max_blocks_per_seq=4)

    def call(q=A, pos=A, group=A, table=A, out=A, ws=A, layer=0, short=0, cache=A, **kw):
        d = _desc(kvc, **dict(base, **kw))
        n = max(kvc.shared_workspace_bytes(d), 1 << 30) if not short else kvc.shared_workspace_bytes(d) - short
        return L.kvc_decode_attention_shared(ctypes.byref(d), cache, layer, q, pos, group, table, None, out, ws, n, None)

    for name in ("cache", "q", "pos", "group", "table", "out", "ws"):
        assert call(**{name: None}) == kvc.KVC_ERR_NULL, name
    for name in ("cache", "q", "out", "ws"):
        assert call(**{name: A + 8}) == kvc.KVC_ERR_ALIGN, name
    assert call(group=A + 2) == kvc.KVC_ERR_ALIGN
    assert call(layer=2) == kvc.KVC_ERR_ARG and call(short=1) == kvc.KVC_ERR_WORKSPACE
    for kw in (dict(dtype="f32"), dict(dtype="i8"), dict(block_size=12), dict(block_size=48), dict(block_size=100),
               dict(q_heads=258)):
        assert call(**kw) == kvc.KVC_ERR_UNSUPPORTED, kw
        assert kvc.shared_workspace_bytes(_desc(kvc, **dict(base, **kw))) == 0
    d = _desc(kvc)
    assert L.kvc_decode_attention_shared(ctypes.byref(d), A, 0, A, A, A, A, None, A, A, 1 << 30, None) == kvc.KVC_ERR_DESC
    assert kvc.shared_workspace_bytes(d) == 0
    with pytest.raises(kvc.KvcError):
        kvc.alloc_shared_workspace(d)
    assert kvc.shared_workspace_bytes(_desc(kvc, **base)) > kvc.workspace_bytes(_desc(kvc, **base))
