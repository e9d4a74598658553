"""4-bit products of one call that name the same tokens with different K.

Bytes of one buffer, read as [M][K] for several K (e4m3): the products are those
of each matrix with its own reading.  Tolerance: test_gpu_fp4.py's.
"""
import numpy as np
import pytest

import draft_helpers as dh
from test_gpu_fp4 import _check, _weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 16, 17, 40, 128])
@pytest.mark.parametrize("Ks", [(128, 640, 256), (640, 128, 640), (256, 1024, 256)], ids=str)
def test_one_buffer_at_several_widths(dev, w12mod, M, Ks):
    import torch
    rng = np.random.default_rng(M + sum(Ks))
    K0 = max(Ks)
    buf = torch.from_numpy((30.0 * rng.standard_normal(M * K0)).astype(np.float32)).to(dev).to(torch.float8_e4m3fn)
    xs = [buf[:M * K].view(M, K) for K in Ks]
    scale = torch.from_numpy(rng.uniform(0.001, 0.02, M).astype(np.float32)).to(dev)
    pairs = [_weight(w12mod, dev, rng, K, 300 - 7 * i, 0.02) for i, K in enumerate(Ks)]
    ys = [torch.full((M, w.N), 5.0, device=dev) for w, _ in pairs]
    ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w for w, _ in pairs], M), dev)
    w12mod.FP4Batch([w for w, _ in pairs], xs, ys, ws, [scale] * len(Ks))()
    for (w, w64), x, y in zip(pairs, xs, ys):
        x64 = dh.bits_f64(x) * scale.cpu().numpy().astype(np.float64)[:, None]
        _check(y, x64, w64, False, (M, w.K, w.N))
    assert w12mod.get_device_error(ws) == w12mod.OK
