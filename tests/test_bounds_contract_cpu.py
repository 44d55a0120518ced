"""What the header says of a block's bounds, on their plain form (which the GPU's codes and steps equal): a code times the
step is outside of the keys, or inside by 2^-23 of the block's largest key at most.

step = a / 127 (1 + d), |d| <= 2^-24, for a >= 127 2^-126.  A code that is not clamped is at least x / step (1 - 2^-24)
for a largest value x > 0: within 2^-24 a; a clamped one gives 127 step >= a (1 - 2^-24).  One of the two roundings counts
for each value, and the product is taken exactly here; 2^-23 leaves room for a product in fp32."""

import pytest
import torch

from tests import part_plain as part


def _excess(k):
    """The largest part of |key| max that lies outside of code * step, over the rows k [rows, D] (fp32 values)."""
    codes, step = part.ends(k)
    top = codes.double() * step.double()
    x = k.double()
    return float(torch.maximum(x.amax(0) - top[0], top[1] - x.amin(0)).max() / x.abs().max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("exponent", [-118, -60, 0, 100])
def test_bounds_hold_to_the_rounding_of_a_step(dtype, exponent):
    g = torch.Generator().manual_seed(exponent + 200)
    beyond, blocks = 0, 600
    for i in range(blocks):
        rows, D = 1 + i % 17, 64
        k = (torch.randn(rows, D, generator=g) * (1 if i % 3 else 3 ** (i % 7))).to(dtype).float() * 2.0 ** exponent
        e = _excess(k)
        assert e <= 2.0 ** -23, i
        beyond += e > 0
    assert beyond > blocks // 4          # (an exact bound would leave none)


def test_signs_and_single_values():
    """Blocks all below or all above zero, with one value, with channels of very different sizes."""
    g = torch.Generator().manual_seed(1)
    for i in range(300):
        k = torch.randn(5, 64, generator=g).abs() * torch.logspace(-30, 3, 64)[torch.randperm(64, generator=g)]
        for x in (k, -k, k[:1], -k[:1], k.clamp(min=k.max())):
            assert _excess(x) <= 2.0 ** -23


def test_steps_below_the_normal_numbers_bound_nothing():
    """Why the header excepts them: a step of 0 has codes 0, and a rounded subnormal step can be off by half of itself."""
    tiny = torch.full((1, 64), 1e-44)
    codes, step = part.ends(tiny)
    assert float(step) == 0.0 and not codes.any()
    assert _excess(torch.full((1, 64), 187 * 2.0 ** -149)) > 2.0 ** -23
