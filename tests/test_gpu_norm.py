"""w12_add_norm against its formula in float64.

Tolerances (u = 2^-24, fp32's half step): h is one addition of fp32 or bf16
numbers, off by u |h|.  The sum of dim squares is added up in chains of at most
32 in a thread and trees of at most 10 more steps, so it is off by less than 64 u
of itself, its root by half of that; with the mean's division, the root, the
reciprocal (1 u each) and the products with weight (its addition of offset, 1 u
of |w| <= 2 |w + offset| here), weight and reciprocal, y is off by less than
(32 + 8) u |y| + u |h w r| < 2^-18 |y| before it is rounded: bf16 adds 2^-8 |y|,
e4m3 half a step of the code (2^-4 of it, at least 2^-10: half of e4m3's smallest
step 2^-9), with the scale's own 2^-18 beside it.
"""
import numpy as np
import pytest

import draft_helpers as dh

pytestmark = pytest.mark.gpu
Y = 2.0 ** -18


def _rows(torch, a, dtype, dev, pad):
    n, dim = a.shape
    t = torch.zeros(n, dim + pad, dtype=torch.float32, device=dev)
    t[:, :dim] = torch.from_numpy(a.astype(np.float32))
    return t.to(dtype)[:, :dim]


def _check_out(torch, out, scale, y, what):
    if scale is None:
        got = dh.bits_f64(out)
        err, tol = np.abs(got - y), np.abs(y) * (2.0 ** -8 + Y) + 1e-38
    else:
        s = scale.cpu().numpy().astype(np.float64)[:, None]
        amax = np.abs(y).max(-1, keepdims=True)
        live = amax > 1.1e-30
        assert np.all(np.abs(s - amax / 448.0)[live] <= (Y * amax / 448.0)[live]), what
        code = dh.bits_f64(out)
        want = np.where(live, y / np.where(live, amax, 1.0) * 448.0, 0.0)
        err, tol = np.abs(code - want), np.abs(want) * (2.0 ** -4 + 2 * Y) + 2.0 ** -10
        assert np.all(s[~live] == 0.0), what
    assert np.all(err <= tol), (what, float((err - tol).max()), np.argwhere(err > tol)[:3])


CASES = [  # n, dim, x f32, delta (None, f32, bf16), weight (None, f32, bf16), offset, e4m3, pad
    (1, 5120, False, "f32", "bf16", 0.0, False, 0),
    (7, 5120, False, "bf16", "f32", 1.0, True, 0),
    (3, 1, True, "f32", None, 0.0, False, 0),
    (2, 1, False, None, "bf16", 0.0, True, 3),
    (5, 33, True, "bf16", "bf16", 1.0, True, 2),
    (300, 1027, False, "f32", "bf16", 0.0, False, 0),
    (40, 2883, True, "f32", "f32", 0.0, True, 5),
    (9, 8192, True, None, "bf16", 1.0, False, 8),
    (6, 8200, False, "f32", "bf16", 0.0, True, 0),   # past 1024 threads of eight
    (4, 8193, False, "bf16", None, 0.5, False, 0),
    (2, 32768, True, "f32", "f32", 0.0, True, 0),
    (2, 32767, False, "f32", "bf16", 0.0, False, 1),
    (1000, 64, False, "bf16", "bf16", 0.0, True, 16),
]


@pytest.mark.parametrize("n,dim,xf,delta,weight,offset,e4m3,pad", CASES)
def test_add_norm(dev, w12mod, n, dim, xf, delta, weight, offset, e4m3, pad):
    import torch
    rng = np.random.default_rng(dim + n)
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}
    x = 2.0 * rng.standard_normal((n, dim))
    x[:, dim // 3] *= 30.0
    if n > 2:
        x[1] *= 1e-12
        x[2] = 0.0
    xt = _rows(torch, x, torch.float32 if xf else torch.bfloat16, dev, pad)
    dt = None if delta is None else _rows(torch, np.where(x[:, :1] == 0, 0.0, rng.standard_normal((n, dim)) * np.abs(x).max(-1, keepdims=True) / 8),
                                          kind[delta], dev, 2 * pad)
    wt = None if weight is None else torch.from_numpy(rng.uniform(0.5, 1.5, dim) * rng.choice([-1, 1], dim) * (1 - offset / 2)).to(kind[weight]).to(dev)
    out = torch.full((n, dim + pad), 7.0, device=dev).to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)[:, :dim]
    res = torch.full((n, dim + pad), 7.0, dtype=xt.dtype, device=dev)
    scale = torch.empty(n, device=dev) if e4m3 else None
    w12mod.add_norm(xt, wt, out, delta=dt, residual_out=res[:, :dim], eps=1e-6, offset=offset, scale_out=scale)
    h, y = dh.add_norm(dh.bits_f64(xt), None if dt is None else dh.bits_f64(dt), None if wt is None else dh.bits_f64(wt), offset, 1e-6)
    err = np.abs(dh.bits_f64(res[:, :dim]) - h)
    assert np.all(err <= np.abs(h) * (2.0 ** -24 if xf else 2.0 ** -8 + 2.0 ** -24))
    _check_out(torch, out, scale, y, (n, dim))
    if pad:  # what lies between the rows stays
        assert bool((res[:, dim:] == 7.0).all())
    # without the residual, and in place of x
    out2 = torch.empty_like(out)
    w12mod.add_norm(xt, wt, out2, delta=dt, offset=offset, scale_out=scale)
    assert torch.equal(out2.float(), out.float())
    w12mod.add_norm(xt, wt, out2, delta=dt, residual_out=xt, offset=offset, scale_out=scale)
    assert torch.equal(out2.float(), out.float()) and torch.equal(xt, res[:, :dim])


def test_large_and_odd_values(dev, w12mod):
    """Rows whose squares pass fp32, and rows with NaN or infinity."""
    import torch
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 96))
    x[0] *= 1e25
    x[1] *= 1e37
    x[2, 5] = np.nan
    x[3, 7] = np.inf
    x[4, 7] = -np.inf
    for dtype in (torch.float32, torch.bfloat16):
        xt = torch.from_numpy(x.astype(np.float32)).to(dtype).to(dev)
        ok = [0, 1, 5]
        _, y = dh.add_norm(dh.bits_f64(xt), None, None, 0.0, 1e-6)
        out = torch.empty(6, 96, dtype=torch.bfloat16, device=dev)
        w12mod.add_norm(xt, None, out)
        _check_out(torch, out[ok], None, y[ok], dtype)
        assert bool(out[2].isnan().all()) and bool(out[3, 7].isnan()) and bool(out[4, 7].isnan())
        codes = torch.empty(6, 96, dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty(6, device=dev)
        w12mod.add_norm(xt, None, codes, scale_out=scale)
        _check_out(torch, codes[ok], scale[ok], y[ok], dtype)
        assert scale.isnan().tolist() == [False, False, True, True, True, False]
        assert bool((codes[2:5].float() == 0).all())


def test_broadcast_rows_other_stream_and_graph(dev, w12mod):
    """Stride 0 inputs, a side stream, a captured call replayed on new values."""
    import torch
    rng = np.random.default_rng(4)
    one = torch.from_numpy(rng.standard_normal((1, 512)).astype(np.float32)).to(dev)
    d = torch.from_numpy(rng.standard_normal((9, 512)).astype(np.float32)).to(dev)
    w = torch.ones(512, device=dev)
    out = torch.empty(9, 512, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w12mod.add_norm(one.expand(9, 512), w, out, delta=d)
    torch.cuda.current_stream().wait_stream(side)
    _, y = dh.add_norm(dh.bits_f64(one), dh.bits_f64(d), None, 0.0, 1e-6)
    _check_out(torch, out, None, y, "side stream")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        w12mod.add_norm(one.expand(9, 512), w, out, delta=d)
    d.mul_(-3.0)
    graph.replay()
    _, y = dh.add_norm(dh.bits_f64(one), dh.bits_f64(d), None, 0.0, 1e-6)
    _check_out(torch, out, None, y, "replay")


def test_refusals(dev, w12mod):
    import torch
    x = torch.zeros(4, 64, device=dev)
    out = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    for bad in (lambda: w12mod.add_norm(x, w[:32], out), lambda: w12mod.add_norm(x, w, out[:3]),
                lambda: w12mod.add_norm(x, w, out, residual_out=out), lambda: w12mod.add_norm(x, w, out.t().contiguous().t()),
                lambda: w12mod.add_norm(x.half(), w, out), lambda: w12mod.add_norm(x.cpu(), w, out)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: w12mod.add_norm(x, w, x), lambda: w12mod.add_norm(x, w, out, scale_out=w[:4].clone()),
                lambda: w12mod.add_norm(x, w, out, eps=-1.0), lambda: w12mod.add_norm(x, w, out, offset=float("nan")),
                lambda: w12mod.add_norm(x, w, out[:1].expand(4, 64))):
        with pytest.raises(w12mod.W12Error):
            bad()
    w12mod.add_norm(x[:0], w, out[:0])


@pytest.mark.parametrize("n,dim", [(5000, 40), (1200, 2883), (700, 5120)])
def test_more_rows_than_ctas_in_place(dev, w12mod, n, dim):
    """A CTA's rows are asked for ahead of the writes of the rows before: in place of x, and of delta."""
    import torch
    rng = np.random.default_rng(dim)
    x = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).to(dev, torch.bfloat16)
    d = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).to(dev, torch.bfloat16)
    h, y = dh.add_norm(dh.bits_f64(x), dh.bits_f64(d), None, 0.0, 1e-6)
    for place in (0, 1):
        a, b = x.clone(), d.clone()
        out = torch.empty(n, dim, dtype=torch.bfloat16, device=dev)
        w12mod.add_norm(a, None, out, delta=b, residual_out=(a, b)[place])
        _check_out(torch, out, None, y, place)
        err = np.abs(dh.bits_f64((a, b)[place]) - h)
        assert np.all(err <= np.abs(h) * (2.0 ** -8 + 2.0 ** -24))
        assert torch.equal((b, a)[place], (d, x)[place])
