"""Draft blocks with many tiles per worker, whose last tiles need a mask, in a
cache whose every unused row is NaN.

Tolerances as in test_gpu_attend.  On e4m3 the fp16 weights' floor has its term:
a weight is off by up to 2^-31 of the row's largest weight times the largest
value scale, so an output by 2^-31 max(scale) max(code) per key.  max(code) is
at most 448, and the row with the largest scale has a code of 90 or more among
its 128 (normal, of deviation 60: all below with probability 1e-8; of 64, 1e-4),
so that product is below 8 max |v|.
"""
import numpy as np
import pytest

from test_gpu_attend import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T", [5, 16])
def test_long_draft_blocks(dev, w12mod, T, e4m3):
    """8 requests of 700 .. 9000 keys, 8 key heads: about 16 tiles a worker; 30
    and 96 query rows, i.e. softmax warps without a valid row, and with one."""
    import torch
    lens = [700 + (9000 - 700) * ((i * 7) % 8) // 7 for i in range(8)]
    p = Problem(w12mod, dev, 8, T, 48, 8, 128, 64, e4m3, lens)
    p.poison()
    out, lse = p.run()
    assert w12mod.get_device_error(p.ws) == 0
    p.check(out, lse, floor=2.0 ** -28 if e4m3 else 0.0)
    for _ in range(20):  # the same bits however the copies fall
        again, z = p.run(ws=p.ws)
        assert torch.equal(out, again) and torch.equal(lse, z)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_one_head_of_small_channels(dev, w12mod, e4m3):
    """64 channels, one key head, requests that end before, at and after a tile's end."""
    p = Problem(w12mod, dev, 6, 9, 4, 1, 64, 32, e4m3, [128 * 40 + n for n in (-3, 0, 4, 5, 120, 131)])
    p.poison()
    out, lse = p.run()
    assert w12mod.get_device_error(p.ws) == 0 and np.isfinite(out.float().cpu().numpy()).all()
    p.check(out, lse, floor=2.0 ** -28 if e4m3 else 0.0)
