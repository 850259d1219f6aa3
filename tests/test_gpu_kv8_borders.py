"""Calls of the 8-bit cache's attention at the borders of what its header allows."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_ref as R  # noqa: E402
from test_gpu_kv8 import D, Pair, spin, step_of  # noqa: E402


@pytest.mark.parametrize("new", [1, 3, 30, 128], ids=["one", "few", "shared", "many"])
@pytest.mark.parametrize("x", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_and_sees_nothing(new, x):
    """Zeros, as for any row that sees nothing; NaN for the head that sees something."""
    p = Pair(1, 2, 2, 8, seed=new)
    p.append([384 - new])
    p.append([new])
    s = p.last[0]
    q = p.rand(new, 4, D)
    q[0, :, 5] = q[new - 1, :, 127] = x
    sel = torch.tensor([[-1, -1, -1], [0, -1, -1]], dtype=torch.int32, device="cuda")
    out = torch.full((new, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    p.c.attend(s, q.cuda(), out, sel=sel)
    got = out.cpu().double()
    assert (got[:, :2] == 0).all()
    assert torch.isnan(got[0, 2:]).all() and torch.isnan(got[-1, 2:]).all()
    assert torch.isfinite(got[1:-1, 2:]).all()
    p.c.check()
