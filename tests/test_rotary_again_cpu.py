"""kvc_rotary_init on a struct that has been through it before: everything follows the fields as they are
now, the magnitude too unless the caller set one."""

import ctypes

import pytest

from tests import plain_ops as plain


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _again(kvc, r, **fields):
    for name, value in fields.items():
        setattr(r, name, value)
    assert kvc.lib().kvc_rotary_init(ctypes.byref(r)) == kvc.KVC_OK
    return r


def _same(kvc, r, **spec):
    fresh = kvc.make_rotary("half", **spec)
    assert r.ready == 1 and list(r.turns[:r.dim // 2]) == list(fresh.turns[:fresh.dim // 2])
    assert r.magnitude == fresh.magnitude
    if not spec.get("magnitude"):
        assert abs(r.magnitude - plain.frequencies(**spec)[1]) <= 2.0 ** -23 * r.magnitude


def test_magnitude_follows_the_fields(kvc):
    yarn = dict(dim=64, scaling="yarn", original_len=4096)
    r = kvc.make_rotary("half", factor=4.0, **yarn)
    _same(kvc, _again(kvc, r), factor=4.0, **yarn)                     # nothing changed
    _same(kvc, _again(kvc, r, factor=32.0), factor=32.0, **yarn)
    _same(kvc, _again(kvc, r, scaling=kvc.SCALINGS["none"]), dim=64)
    _same(kvc, _again(kvc, r, scaling=kvc.SCALINGS["yarn"], factor=8.0, original_len=2048), dim=64, scaling="yarn",
          original_len=2048, factor=8.0)


def test_a_callers_magnitude_stays(kvc):
    yarn = dict(dim=64, scaling="yarn", original_len=4096)
    r = kvc.make_rotary("half", factor=4.0, magnitude=0.75, **yarn)
    _same(kvc, _again(kvc, r, factor=16.0), factor=16.0, magnitude=0.75, **yarn)
    r = _again(kvc, kvc.make_rotary("half", factor=4.0, **yarn), magnitude=2.0)     # set after a first call
    assert r.magnitude == 2.0
    _same(kvc, _again(kvc, r, factor=16.0), factor=16.0, magnitude=2.0, **yarn)
    _same(kvc, _again(kvc, r, magnitude=0.0), factor=16.0, **yarn)     # and given back


def test_after_a_refusal(kvc):
    r = kvc.make_rotary("half", dim=64, scaling="yarn", original_len=4096, factor=4.0)
    r.factor = -1.0
    assert kvc.lib().kvc_rotary_init(ctypes.byref(r)) == kvc.KVC_ERR_ARG and r.ready == 0
    _same(kvc, _again(kvc, r, factor=64.0), dim=64, scaling="yarn", original_len=4096, factor=64.0)
