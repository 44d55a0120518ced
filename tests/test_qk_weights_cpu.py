"""The norm weights that a kvc_qk carries are checked by every call that uses it: they may have been
given with another descriptor, or lie on another device."""

import pytest
import torch


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _qk(kvc, q=None, k=None):
    qk = kvc.KvcQk(None, 1 << 20 if q is not None else None, 1 << 20 if k is not None else None, 1e-6, 0.0)
    qk.keep = (None, q, k)
    return qk


def _call(kvc, qk, head_dim=128, dtype="bf16"):
    d = kvc.make_desc("ring", "none", dtype, layers=1, batch=3, q_heads=8, kv_heads=2, head_dim=head_dim, window=100)
    x = torch.zeros(3, 8, head_dim, dtype=kvc.desc_dtype(d))
    kvc.append_qk(d, x, 0, x, x, x, x, x, qk)


@pytest.mark.parametrize("side", ["q", "k"])
def test_weights_of_another_descriptor(kvc, side):
    """Refused for the weights before anything else (the call's other tensors are no CUDA tensors either)."""
    bf16 = lambda n: torch.zeros(n, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=side + "_weight must have 128 elements"):
        _call(kvc, _qk(kvc, **{side: bf16(64)}))
    with pytest.raises(TypeError, match=side + "_weight must be torch.float32"):
        _call(kvc, _qk(kvc, **{side: bf16(128)}), dtype="f32")
    with pytest.raises(TypeError, match=side + "_weight must be torch.bfloat16"):
        _call(kvc, _qk(kvc, **{side: torch.zeros(128)}), dtype="i8")
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        _call(kvc, _qk(kvc, **{side: bf16(128)}))


def test_weights_of_another_device(kvc):
    d = kvc.make_desc("ring", "none", "bf16", layers=1, batch=3, q_heads=8, kv_heads=2, head_dim=128, window=100)
    w = torch.zeros(128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_weight is on"):
        kvc._need_qk(kvc._sizes_of(d), _qk(kvc, k=w), 0)


@pytest.mark.gpu
def test_refused_before_any_launch(kvc):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    descs = {D: kvc.make_desc("ring", "none", "bf16", layers=1, batch=2, q_heads=4, kv_heads=2, head_dim=D, window=8)
             for D in (64, 128)}
    small = kvc.make_qk(descs[64], q_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    d = descs[128]
    cache, ws = kvc.alloc_cache(d, fill=3.0), kvc.alloc_workspace(d)
    q, k, v = (torch.ones(2, n, 128, dtype=torch.bfloat16, device="cuda") for n in (4, 2, 2))
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="q_weight"):
        kvc.append_qk(d, cache, 0, q, k, v, pos, ws, small)
    assert bool((cache == 3.0).all())
