"""4-bit products whose sums have one sign, over long K.

The tensor core cuts where it adds, so a sum of one sign drifts with the number
of additions it is made of.  Tolerance: one step adds 16 products to a running
sum; if it loses less than 2 2^-23 of that sum (its last place and the products'
cuts; 8192 steps in a row lost 5e-4, 2^-23 each), which rises evenly over the 512
steps (8192 k) of a part, a part is off by less than 512 / 2 2 2^-23 = 2^-14 of
itself; up to 16 parts are added in fp32, the scales' products are 3 2^-24.  Below
2^-13.7 of the sum.
"""
import numpy as np
import pytest

import draft_helpers as dh

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -13.7


def _positive(w12mod, dev, rng, K, N):
    """A matrix of eight different columns of positive weights, over and over."""
    import torch
    codes = (rng.integers(0, 8, (8, K // 2)) | rng.integers(0, 8, (8, K // 2)) << 4).astype(np.uint8)
    scales = rng.integers(0x30, 0x40, (8, K // 16)).astype(np.uint8)
    c = torch.from_numpy(codes).to(dev).repeat((N + 7) // 8, 1)[:N].contiguous()
    s = torch.from_numpy(scales).to(dev).repeat((N + 7) // 8, 1)[:N].contiguous()
    return w12mod.FP4Weight.pack(c, s.view(torch.float8_e4m3fn), 0.01), dh.fp4_values(codes, scales, 0.01)


@pytest.mark.parametrize("M", [5, 17, 33, 65, 128])
@pytest.mark.parametrize("K,tiles", [(1024, 3), (5120, 136), (17408, 160), (131072, 152)])
def test_sums_of_one_sign(dev, w12mod, M, K, tiles):
    import torch
    rng = np.random.default_rng(M + K)
    N = 256 * tiles - 3
    w, w64 = _positive(w12mod, dev, rng, K, N)
    x = torch.from_numpy(rng.uniform(0.5, 1.0, (M, K)).astype(np.float32)).to(dev, torch.bfloat16)
    want = dh.bits_f64(x) @ w64.T
    y = torch.empty(M, N, device=dev)
    ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w], M), dev)
    w12mod.fp4_gemm(w, x, y, ws)
    got = y.double()
    ref = torch.from_numpy(want).to(dev).repeat(1, (N + 7) // 8)[:, :N]
    off = ((got - ref) / ref)
    print(f"M {M} K {K}: mean {float(off.mean()):.2e} largest {float(off.abs().max()):.2e}")
    assert float(off.abs().max()) <= TOL
    assert w12mod.get_device_error(ws) == w12mod.OK
