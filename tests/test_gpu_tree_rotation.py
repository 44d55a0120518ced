"""kvc_tree_attention with rotated keys, against float64 whose rotated rows are rounded as the cache stores them: a query or
a drafted key at any other position than its own is seen (test_draft_plain_cpu.py shows that of the tolerances)."""

import pytest
import torch

from tests.test_gpu_tree_segments import Batch, kvc  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["paged", "ring", "sink_ring"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 12, 33, 64])
def test_positions_of_rotated_rows(kvc, layout, D, T):  # noqa: F811
    lens = [150, 131, 260, 64, 0, 1]
    kw = {} if layout == "paged" else dict(window=100, sinks=4 if layout == "sink_ring" else 0)
    s = Batch(kvc, layout, lens, T, 8, 2, D, "baked", **kw)
    out = s.run()
    assert kvc.get_error(s.ws) == 0
    s.check(out)
    s.repeat(out, 5)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_far_positions(kvc, D):  # noqa: F811
    """Rings far along: the angle of a position is reduced exactly."""
    s = Batch(kvc, "ring", [10 ** 6 + 7, 70, 3 * 10 ** 5], 20, 4, 2, D, "baked", window=64)
    s.check(s.run())


@pytest.mark.parametrize("H,KV", [(12, 4), (10, 2), (32, 1)])
def test_positions_of_head_groups(kvc, H, KV):  # noqa: F811
    s = Batch(kvc, "paged", [150, 90, 33], 24, H, KV, 128, "baked")
    out = s.run()
    s.check(out)
    s.repeat(out, 5)
