"""FP4Weight.encode's own scale: of the finite weights, on the given stream."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _weights(rng, N, K):
    import torch
    return torch.from_numpy((0.02 * rng.standard_normal((N, K))).astype(np.float32)).to(torch.bfloat16)


def test_one_bad_weight_moves_no_other_group(dev, w12mod):
    import torch
    rng = np.random.default_rng(1)
    w = _weights(rng, 9, 256)
    w[4, 7] = 0.5  # the largest, in a group that stays
    clean = w12mod.FP4Weight.encode(w.to(dev))
    for bad in (float("nan"), float("inf"), float("-inf")):
        v = w.clone()
        v[2, 35] = bad
        enc = w12mod.FP4Weight.encode(v.to(dev))
        assert enc.scale == clean.scale == 0.5 / 2688.0 or abs(enc.scale * 2688.0 - 0.5) < 1e-6
        a, b = enc.decode().cpu(), clean.decode().cpu()
        assert bool(a[2, 32:48].isnan().all()) if bad != bad else bool(a[2, 32:48].isfinite().all())
        keep = torch.ones(9, 256, dtype=torch.bool)
        keep[2, 32:48] = False
        assert torch.equal(a[keep], b[keep])


def test_nothing_finite_and_tiny_weights(dev, w12mod):
    import torch
    w = torch.full((2, 128), float("nan"), dtype=torch.bfloat16)
    assert bool(w12mod.FP4Weight.encode(w.to(dev)).decode().isnan().all())
    assert bool((w12mod.FP4Weight.encode(torch.zeros(2, 128, dtype=torch.bfloat16, device=dev)).decode() == 0).all())
    # below 2^-88 the scale is the smallest one, 2^-100, and the groups' scales are smaller than 448:
    # half a step of 6 codes of the largest, and of a group's scale (3 bits: 2^-4)
    w = (1e-29 * torch.from_numpy(np.random.default_rng(2).uniform(0.9, 1.0, (3, 128)).astype(np.float32))).to(torch.bfloat16)
    enc = w12mod.FP4Weight.encode(w.to(dev))
    assert enc.scale == 2.0 ** -100
    v = w.double()
    assert bool(((enc.decode().cpu().double() - v).abs() <= v.abs().max() * (1 / 6 + 1 / 16)).all())


def test_scale_is_of_the_stream_given(dev, w12mod):
    """The weights are written on the stream that is named; the current stream knows nothing of it."""
    import torch
    rng = np.random.default_rng(3)
    src = _weights(rng, 64, 1024).to(dev)
    want = w12mod.FP4Weight.encode(src)
    side = torch.cuda.Stream()
    big = torch.randn(6144, 6144, device=dev)
    w = torch.full_like(src, 100.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):
            big = (big @ big).clamp(-1, 1)
        w.copy_(src)
    enc = w12mod.FP4Weight.encode(w, stream=side)
    side.synchronize()
    assert enc.scale == want.scale
    assert torch.equal(enc.decode().cpu(), want.decode().cpu())
    del big
