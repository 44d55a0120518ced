"""The tolerances of the drafted tokens' tests tell a rotation at a wrong position from a right one (CPU)."""

import pytest
import torch

from tests import draft_plain as draft


def _case(D, n, T, seed):
    g = torch.Generator().manual_seed(seed)
    H, KV = 8, 2
    # (sizes as the GPU tests draw them: q of 0.75, keys and values of 1)
    q = (torch.randn(T, H, D, generator=g) * 0.75).to(torch.bfloat16).double()
    k, v, kc, vc = (torch.randn(m, KV, D, generator=g).to(torch.bfloat16).double() for m in (T, T, n, n))
    return (q, k, v, draft.random_tree(T, seed), n, list(range(n)), kc, vc, "paged", 0, 0, D ** -0.5, "baked")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [64, 131, 260])
@pytest.mark.parametrize("T", [12, 33])
def test_misplaced_rotations_are_seen(D, n, T):
    args = _case(D, n, T, D + n + T)
    tok, want, tol = draft.attend(*args)
    assert tok == list(range(T))
    draft.compare(want.to(torch.bfloat16), T, tok, want, tol)
    for plant in ("q one further", "keys at pos0", "keys as they came"):
        _, other, _ = draft.attend(*args, plant=plant)
        err = ((other - want).abs() / tol).amax((1, 2))
        if plant == "keys at pos0":          # (seen by tokens that attend a deeper one, itself among them)
            assert sum(float(e) > 1 for e in err) >= T // 4, plant
        else:
            assert (err > 1).all(), plant
        with pytest.raises(AssertionError):
            draft.compare(other.to(torch.bfloat16), T, tok, want, tol)


def test_only_values_at_a_tie_are_allowed_for():
    """A rotated value's allowance is 0, or no more than a step of bf16 beside the fp32 error; hardly any has one."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(500, 2, 128, generator=g).to(torch.bfloat16).double()
    y, off = draft.rotated(x, torch.arange(500))
    assert float((off > 0).double().mean()) < 3e-3
    some = off > 0
    assert (off[some] <= 2.0 ** -7 * (y.abs()[some] + 1e-5) + 1e-5).all()
