"""w12_fp4_encode's rounding, as the header states it: fp32 arithmetic
  s = the e4m3 number nearest to round(max |w| / round(6 scale)),
  r = round(1 / round(s scale)), the code nearest to round(|w| r).
Exactly that (a restatement in numpy's fp32), and against the real numbers: an
e2m1 code's argument is off by three roundings, 3 2^-24 of it, so the code is the
nearest one, or |w| lies within 2^-22 (relative) of the middle between the two.
"""
import numpy as np
import pytest

import draft_helpers as dh

pytestmark = pytest.mark.gpu


def _bf16_around(v):
    """The bf16 numbers nearest to v and two to either side."""
    b = np.asarray(v, np.float32).view(np.uint32) >> 16
    return ((b[..., None] + np.arange(-2, 3)).astype(np.uint32) << 16).view(np.float32)


@pytest.mark.parametrize("scale", [1.0, 0.01, 1.0 / 896.0, 2.0 ** -100, 2.0 ** 90], ids=str)
def test_weights_at_the_middles(dev, w12mod, scale):
    import torch
    scale = float(np.float32(scale))
    s = dh.e4m3_values()[1:127]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    # a group: its largest weight, 6 s scale, and the weights around three middles
    rows = []
    for k in range(0, 7, 3):
        m = mids[[k, min(k + 1, 6), min(k + 2, 6)]]
        near = _bf16_around((s * scale)[:, None] * m).reshape(len(s), 15)
        rows.append(np.concatenate([_bf16_around(6.0 * s * scale)[:, 2:3], near], 1))
    g = np.concatenate(rows).astype(np.float32)          # [3 * 126, 16]
    g = np.concatenate([g, np.zeros((-len(g) % 8, 16), np.float32)])
    v = g.reshape(-1, 128) * np.random.default_rng(0).choice([-1.0, 1.0], (len(g) // 8, 128)).astype(np.float32)
    w = torch.from_numpy(v).to(torch.bfloat16)
    assert np.array_equal(w.float().numpy(), v)
    got = w12mod.FP4Weight.encode(w.to(dev), scale).decode().cpu().numpy().astype(np.float64)
    code, sc = dh.fp4_encode(v, scale)
    code = np.where(v < 0, code | 8, code).astype(np.uint8)
    want = dh.fp4_values(code[:, 0::2] | code[:, 1::2] << 4, sc, scale)
    assert np.array_equal(got, want.astype(np.float32))
    # the real numbers, from the definition
    unit = np.repeat(dh.e4m3_values()[sc] * scale, 16, axis=-1)
    err = np.abs(np.abs(got) - np.abs(v))
    best = np.abs(np.abs(v)[..., None] - dh.E2M1 * unit[..., None]).min(-1)
    assert np.all(err <= best + 2.0 ** -21 * np.abs(v) + 1e-44)
