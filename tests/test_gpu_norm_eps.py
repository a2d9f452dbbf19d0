"""Layer norm with a small eps: rows without spread, as padding has them, and rows of little
spread, whose rstd is large.  Tolerances are those of test_gpu_norm.py: all are relative to
terms that scale with rstd.  Spreads are such that their squares are normal fp32 numbers."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gb300 as moe
from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu

WIDTHS = [3, 128, 500, 1001, 2048, 7168, 8200, 16384]   # every shape, with and without a ring


@pytest.mark.parametrize("types", N.TYPES, ids=str)
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("eps", [1e-12, 1e-26, 1e-30, 1e-36])
def test_rows_without_spread(H, types, eps):
    """Rows of zeros and of one value; the mean of H equal powers of two is exact, as are the
    distances of zero from it.  With a spread of sqrt(eps) beside them."""
    eps = float(np.float32(eps))
    d = N.make(40, H, *types)
    h = d["x"].float() * (eps ** 0.5)
    h[0], h[5], h[17], h[39] = 0.0, 1.0, -(2.0 ** 20), 2.0 ** -40
    h = h.to(types[0])
    y, same, stats = moe.moe_layer_norm(h, d["weight"], d["bias"], eps)
    N.check_forward(dict(d, x=h), y, h, stats, eps)
    for row in (0, 5, 17, 39):
        assert torch.equal(y[row], d["bias"].to(y.dtype))
    for dh in (None, d["dh"]):
        got = moe.moe_layer_norm_backward(d["dy"], h, stats, d["weight"], dh=dh)
        assert all(torch.isfinite(t).all() for t in got)
        N.check_backward(d, h, stats, got, dh)
