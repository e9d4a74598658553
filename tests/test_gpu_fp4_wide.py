"""4-bit products of one matrix with more column tiles than the GPU has places
for CTAs: several whole tiles a CTA (an output layer's form).  Tolerance:
test_gpu_fp4.py's."""
import numpy as np
import pytest

from test_gpu_fp4 import _check, _weight, _x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,e4m3", [(1, False), (8, True), (16, False), (17, True), (64, False), (128, False)])
@pytest.mark.parametrize("K,N", [(256, 151936), (384, 80001)])
def test_more_tiles_than_places(dev, w12mod, M, e4m3, K, N):
    import torch
    rng = np.random.default_rng(M + K)
    w, w64 = _weight(w12mod, dev, rng, K, N, 0.01)
    x, xs, x64 = _x(dev, rng, M, K, e4m3)
    ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w], M), dev)
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((M, N), 7.0, dtype=dtype, device=dev)
        w12mod.fp4_gemm(w, x, y, ws, xs)
        _check(y, x64, w64, dtype is torch.bfloat16, (M, K, N))
    assert w12mod.get_device_error(ws) == w12mod.OK
