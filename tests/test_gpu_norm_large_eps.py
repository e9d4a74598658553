"""w12_add_norm with eps as large as the largest squares.

Tolerances: test_gpu_norm.py's.
"""
import numpy as np
import pytest

import draft_helpers as dh
from test_gpu_norm import _check_out
from test_gpu_norm_eps import DIMS, _rows, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("eps", [1e30, 1e37, 3.4e38])
def test_large_eps(dev, w12mod, dim, eps):
    """eps beside squares that pass fp32, and beside small ones."""
    import torch
    rng = np.random.default_rng(dim + 2)
    x = torch.from_numpy(_rows(rng, dim, [1.0, 1e10, 1e15, 1e18, 1e19, 3e19, 1e20, 1e25, 1e36]).astype(np.float32)).to(dev)
    out, codes, scale = _run(w12mod, dev, x, None, eps)
    _, y = dh.add_norm(dh.bits_f64(x), None, None, 0.0, float(np.float32(eps)))
    _check_out(torch, out, None, y, (dim, eps))
    _check_out(torch, codes, scale, y, (dim, eps))
