"""Sampling with temperatures at the ends of their range."""
import numpy as np
import pytest

from test_gpu_sample import Call, _dev

pytestmark = pytest.mark.gpu

TINY = [1e-45, 1e-39, 2.0 ** -128, 2.9e-39, 1.2e-38, 1e-30]


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 4099, 151936])
@pytest.mark.parametrize("cut", ["none", "top_k", "many", "top_p", "min_p"])
def test_smallest_temperatures(dev, w12mod, V, cut, bf16):
    """Any temperature above 0 draws among the largest logits alone, however
    small it is: one of them with probability 1, of three equal ones the u-th
    third."""
    import torch
    n = 2 * len(TINY)
    rng = np.random.default_rng(V)
    x = rng.standard_normal((n, V)).astype(np.float32)
    top = np.array([np.sort(rng.choice(V, 3, replace=False)) for _ in range(n)])
    for r in range(n):
        x[r, top[r, :1 if r < len(TINY) else 3]] = 9.0
    xd = _dev(x, dev)
    xd = xd.to(torch.bfloat16) if bf16 else xd
    u = rng.random(n).astype(np.float32)
    args = {"none": {}, "top_k": dict(top_k=[3] * n), "many": dict(top_k=[min(V - 1, 3000)] * n),
            "top_p": dict(top_p=[0.9999] * n), "min_p": dict(min_p=[0.5] * n)}[cut]
    c = Call(w12mod, dev, xd, n, 1, u, [np.float32(t) for t in TINY] * 2, **args)
    for r in range(n):
        m = 1 if r < len(TINY) else 3
        want = top[r, int(np.floor(np.floor(float(u[r]) * 2.0 ** 24) * m / 2.0 ** 24))]
        assert c.tok[r] == want and abs(c.pr[r] * m - 1.0) <= 2.0 ** -22, r


def test_infinite_temperature(dev, w12mod):
    """All logits above -infinity alike."""
    V = 20000
    x = np.linspace(-50, 50, V, dtype=np.float32)[None].repeat(3, 0)
    x[:, ::4] = -np.inf
    u = np.array([0.0, 0.4, 0.99], dtype=np.float32)
    live = np.nonzero(np.isfinite(x[0]))[0]
    c = Call(w12mod, dev, _dev(x, dev), 3, 1, u, [np.inf] * 3)
    assert c.tok.tolist() == [int(live[int(np.floor(float(a) * 2.0 ** 24)) * len(live) >> 24]) for a in u]
    assert np.all(np.abs(c.pr * len(live) - 1.0) <= 2.0 ** -22)


@pytest.mark.parametrize("V", [7, 151936])
def test_parameters_that_are_nan(dev, w12mod, V):
    """A top_p or min_p that is NaN is no cut (only top_p < 1 and min_p > 0 are
    one); a temperature that is NaN is the greedy choice."""
    rng = np.random.default_rng(V)
    x = _dev(rng.standard_normal((4, V)).astype(np.float32), dev)
    u = rng.random(4).astype(np.float32)
    nan = [float("nan")] * 4
    plain = Call(w12mod, dev, x, 4, 1, u, [1.0] * 4)
    assert plain.tok.tolist() != np.argmax(x.cpu().numpy(), -1).tolist()
    for kw in (dict(top_p=nan), dict(min_p=nan), dict(top_p=nan, min_p=nan, top_k=[0] * 4)):
        c = Call(w12mod, dev, x, 4, 1, u, [1.0] * 4, **kw)
        assert c.tok.tolist() == plain.tok.tolist() and c.pr.tolist() == plain.pr.tolist(), kw
    c = Call(w12mod, dev, x, 4, 1, u, nan)
    assert c.tok.tolist() == np.argmax(x.cpu().numpy(), -1).tolist() and c.pr.tolist() == [1.0] * 4
