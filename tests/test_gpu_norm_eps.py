"""w12_add_norm with eps 0 and very small: rows whose squares are below fp32's
smallest numbers.

Tolerances: test_gpu_norm.py's (the rows are scaled by powers of two, which
rounds nothing but squares and eps far below the others).  A row of zeros with
eps 0 gives zeros.
"""
import numpy as np
import pytest

import draft_helpers as dh
from test_gpu_norm import _check_out

pytestmark = pytest.mark.gpu

DIMS = [1, 96, 1027, 8200]  # by eights, one by one, more than 8192


def _rows(rng, dim, magnitudes):
    x = rng.standard_normal((len(magnitudes), dim)) + 0.1
    return x * np.asarray(magnitudes)[:, None]


def _run(w12mod, dev, x, weight, eps, **kw):
    """(bf16 out), (e4m3 codes, scales) of fp32 rows."""
    import torch
    n, dim = x.shape
    out = torch.empty(n, dim, dtype=torch.bfloat16, device=dev)
    codes, scale = torch.empty(n, dim, dtype=torch.float8_e4m3fn, device=dev), torch.empty(n, device=dev)
    w12mod.add_norm(x, weight, out, eps=eps, **kw)
    w12mod.add_norm(x, weight, codes, eps=eps, scale_out=scale, **kw)
    return out, codes, scale


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-30, 1e-12])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_small_rows(dev, w12mod, dim, eps, kind):
    import torch
    rng = np.random.default_rng(dim)
    mags = [1e-43, 1e-38, 1e-30, 1e-25, 3e-23, 1e-20, 1e-16, 1e-15, 1e-12, 1.0, 1e15]
    x = torch.from_numpy(_rows(rng, dim, mags).astype(np.float32)).to(dev)
    x[:, 0] = torch.tensor(mags, device=dev).float()  # (no row is all zeros, also after rounding)
    if kind == "bf16":
        x = x.to(torch.bfloat16)
    w = torch.from_numpy(rng.uniform(0.5, 1.5, dim).astype(np.float32)).to(dev)
    out, codes, scale = _run(w12mod, dev, x, w, eps)
    h, y = dh.add_norm(dh.bits_f64(x), None, dh.bits_f64(w), 0.0, float(np.float32(eps)))
    y[~h.any(-1)] = 0.0  # (1e-43 is 0 in bf16)
    _check_out(torch, out, None, y, (dim, eps))
    _check_out(torch, codes, scale, y, (dim, eps))


@pytest.mark.parametrize("dim", DIMS)
def test_small_rows_with_delta_and_residual(dev, w12mod, dim):
    """A row's own sum decides, not its parts': x and delta that nearly cancel."""
    import torch
    rng = np.random.default_rng(dim + 1)
    x = torch.from_numpy(_rows(rng, dim, [1e-3, 1e-20, 1e-3]).astype(np.float32)).to(dev)
    d = -x
    d[0] += torch.from_numpy((1e-9 * (1.0 + rng.random(dim))).astype(np.float32)).to(dev)
    d[1] *= 1.0 + 2.0 ** -20
    out = torch.empty(3, dim, dtype=torch.bfloat16, device=dev)
    res = torch.empty_like(x)
    w12mod.add_norm(x, None, out, delta=d, residual_out=res, eps=0.0)
    h = x + d  # (one rounding, as the call's)
    assert torch.equal(res, h)
    _, y = dh.add_norm(dh.bits_f64(h[:2]), None, None, 0.0, 0.0)
    _check_out(torch, out[:2], None, y, dim)
    assert bool((out[2] == 0).all())  # x = -delta: zeros


@pytest.mark.parametrize("dim", DIMS)
def test_zero_rows_without_eps(dev, w12mod, dim):
    """Nothing to divide by: zeros, scale 0; the rows beside it are as they were."""
    import torch
    x = torch.ones(3, dim, device=dev)
    x[1] = 0.0
    out, codes, scale = _run(w12mod, dev, x, None, 0.0)
    assert bool((out[1] == 0).all()) and bool((out[[0, 2]] == 1).all())
    assert bool((codes[1].float() == 0).all()) and scale.tolist()[1] == 0.0 and bool((codes[[0, 2]].float() == 448.0).all())
