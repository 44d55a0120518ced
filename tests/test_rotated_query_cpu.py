"""The tolerances of the rotated queries' tests tell a query at a wrong position from a right one (CPU)."""

import pytest
import torch

from tests import rotated_query as rotated


@pytest.mark.parametrize("dtype", ["bf16", "i8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [40, 150, 700])
def test_misplaced_queries_are_seen(dtype, D, n):
    g = torch.Generator().manual_seed(D + n)
    q = torch.randn(4, D, generator=g).to(torch.bfloat16).double()
    k, v = (torch.randn(n, D, generator=g).to(torch.bfloat16).double() for _ in range(2))
    want, tol, w, _ = rotated.attend(q, n - 1, k, v, D ** -0.5, dtype)
    assert ((want.to(torch.bfloat16).double() - want).abs() <= tol).all()
    for t in (n, n - 2, 0):
        other, _, u, _ = rotated.attend(q, t, k, v, D ** -0.5, dtype)
        assert (((other - want).abs() / tol).amax(-1) > 1).all(), t
        assert float((u - w).abs().max() / w.max()) > 0.02
