"""The paged cache on the GPU: append (rotary positions, rounding or
quantisation) and read-back against plain 64-bit forms.

Tolerances.  A rotated channel is two fp32 products and a sum of values that
are exact in fp32, with the table's cos and sin rounded to fp32: the error is
below 4 * 2^-24 (|x| + |y|) for the pair (x, y).  bf16 then rounds by at most
2^-8 of the value (8 significant bits).  An e4m3 code of z = x / scale is the nearest multiple of
2^-9 (subnormal) or has a relative error of 2^-4; z carries the fp32 errors
of the scale, its reciprocal and the product (3 * 2^-24 relative).
"""
import numpy as np
import pytest

from step_helpers import cache_values, pages, request_rows, rotate

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def _dev(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _fill(kv, rng):
    """Bytes of a used cache: anything, NaN codes included."""
    import torch
    for t in (kv.k, kv.v):
        n = t.numel() * t.element_size()
        t.view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 256, n, dtype=np.uint8)).view(
            t.view(torch.uint8).shape))
    for t in (kv.k_scale, kv.v_scale):
        if t is not None:
            t.fill_(float("nan"))


def _raw(kv):
    import torch
    return [t.contiguous().view(torch.uint8).cpu().numpy().copy()
            for t in (kv.k, kv.v, kv.k_scale, kv.v_scale) if t is not None]


def _tol(x, y, rot, interleaved):
    """fp32 error bound of the rotated channels (0 for those left alone)."""
    t = np.zeros_like(x)
    if rot:
        i0 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
        i1 = i0 + 1 if interleaved else i0 + rot // 2
        b = 4 * EPS * (np.abs(x[..., i0]) + np.abs(x[..., i1]))
        t[..., i0] = b
        t[..., i1] = b
    return t


CASES = [  # R, T, hq, hkv, dim, rot, interleaved, page, e4m3, f32, lens
    (1, 1, 1, 1, 128, 128, False, 16, False, False, [1]),
    (1, 1, 6, 1, 128, 128, False, 64, True, True, [700]),
    (3, 5, 12, 2, 128, 64, True, 32, True, False, [5, 37, 1000]),
    (4, 3, 4, 4, 64, 64, False, 128, False, True, [3, 4, 130, 257]),
    (2, 17, 3, 1, 64, 24, False, 16, True, True, [17, 33]),
    (2, 4, 5, 5, 64, 40, True, 16, False, False, [9, 16]),
    (2, 4, 2, 2, 128, 8, False, 64, True, False, [64, 65]),
    (2, 300, 48, 8, 128, 128, False, 64, True, False, [300, 811]),   # four rows in flight per group
    (1, 700, 32, 8, 64, 0, False, 32, False, True, [900]),           # no rotation
    (5, 4, 6, 2, 128, 128, False, 16, True, False, [0, 1, 3, 4, 18]),  # padding tokens
    (1, 4093, 12, 2, 128, 96, True, 64, True, True, [4093]),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c[:10]).replace(" ", "") for c in CASES])
def test_append(dev, w12mod, case):
    import torch
    R, T, hq, hkv, dim, rot, inter, page, e4m3, f32, lens = case
    rng = np.random.default_rng(R * 1000 + T * 10 + dim + rot)
    table, n_pages = pages(rng, lens, page)
    kv = w12mod.KVCache.alloc(n_pages, hkv, dim, page, w12mod.KV_E4M3 if e4m3 else w12mod.KV_BF16, dev)
    _fill(kv, rng)
    before = _raw(kv)
    n = R * T
    x = rng.standard_normal((n, hq + 2 * hkv + 1, dim)).astype(np.float32)  # one more head: a wider token stride
    x[:, hq] *= 30.0
    x = _dev(x, dev)
    x = x if f32 else x.to(torch.bfloat16)
    xs = x.float().cpu().numpy().astype(np.float64)
    rope = _dev(w12mod.rope_table(max(max(lens), 1), rot), dev) if rot else None
    q_out = torch.full((n, hq, dim), 7.0, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    w12mod.kv_append(kv, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv], _dev(table, dev),
                     _dev(np.array(lens, np.int32), dev), T, q_out, rope,
                     w12mod.ROPE_INTERLEAVED if inter else w12mod.ROPE_HALF, err)
    assert int(err.item()) == 0
    pos = np.concatenate([np.arange(m - T, m) for m in lens])
    live = pos >= 0
    # queries
    want = rotate(xs[:, :hq], pos, rot, inter)
    got = q_out.float().cpu().numpy().astype(np.float64)
    tol = _tol(xs[:, :hq], want, rot, inter)
    assert np.all(np.abs(got - want)[live] <= (2.0 ** -8 * (np.abs(want) + tol) + tol)[live])
    assert np.all(got[~live] == 7.0)
    # keys and values
    tok = np.nonzero(live)[0]
    req = tok // T
    pg, row = table[req, pos[tok] // page], pos[tok] % page
    for n_, (new, cached) in enumerate(zip((rotate(xs[:, hq:hq + hkv], pos, rot, inter),
                                            xs[:, hq + hkv:hq + 2 * hkv]), cache_values(kv))):
        new, cached = new[tok], cached[pg, :, row]
        tol = _tol(xs[tok, hq:hq + hkv], new, rot, inter) if n_ == 0 else np.zeros_like(new)
        if e4m3:
            scale = np.abs(new).max(-1, keepdims=True) / 448.0
            rel = 8 * EPS
            tol = np.maximum(2.0 ** -4 * np.abs(new), 2.0 ** -10 * scale) * (1 + rel) + rel * np.abs(new) + 2 * tol
            sc = (kv.k_scale, kv.v_scale)[n_].cpu().numpy()[pg, :, row].astype(np.float64)
            assert np.all(np.abs(sc - scale[..., 0]) <= 8 * EPS * scale[..., 0])
        else:
            tol = 2.0 ** -8 * (np.abs(new) + tol) + tol
        assert np.all(np.abs(cached - new) <= tol)
    # every other byte of the cache is what it was
    after = _raw(kv)
    for a, b in zip(before, after):
        a, b = (y.reshape(n_pages, hkv, page, -1).copy() for y in (a, b))
        a[pg, :, row] = 0
        b[pg, :, row] = 0
        assert np.array_equal(a, b)


def test_append_odd_rows_e4m3(dev, w12mod):
    """All-zero rows, rows too small to scale, rows with a NaN or an infinity."""
    import torch
    dim, T = 128, 6
    x = np.ones((T, 3, dim), dtype=np.float32)
    x[0] = 0.0
    x[1] = 1e-31
    x[2, :, 5] = np.nan
    x[3, :, 100] = -np.inf
    x[4, :, 7] = 1e38
    x[5] = -np.float32(2.0) ** -90
    kv = w12mod.KVCache.alloc(1, 1, dim, 16, w12mod.KV_E4M3, dev)
    q_out = torch.empty((T, 1, dim), dtype=torch.bfloat16, device=dev)
    xd = _dev(x, dev)
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    w12mod.kv_append(kv, xd[:, :1], xd[:, 1:2], xd[:, 2:], table, torch.tensor([T], dtype=torch.int32, device=dev),
                     T, q_out)
    k = torch.empty((T, 1, dim), dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    w12mod.kv_read(kv, table, torch.tensor([0, T], dtype=torch.int32, device=dev), k, v)
    for got in (k.float().cpu().numpy()[:, 0], v.float().cpu().numpy()[:, 0]):
        assert np.all(got[0] == 0.0) and np.all(got[1] == 0.0)
        assert np.all(np.isnan(got[2])) and np.all(np.isnan(got[3]))
        assert abs(got[4, 7] / 1e38 - 1) < 2.0 ** -8 and np.all(got[4, :7] == 0.0)
        assert np.all(np.abs(got[5] * 2.0 ** 90 + 1) <= 2.0 ** -8)


def test_append_bad_entries(dev, w12mod):
    """A page outside the cache, a position past the table or past the rotary
    table: the token writes nothing, the others do, and the error is told."""
    import torch
    dim, page, T = 64, 16, 2
    lens = [18, 18, 40, 18, 9]
    table = np.array([[0, 1], [2, 99], [3, 4], [5, -1], [6, 0]], dtype=np.int32)
    for rope_positions in (64, 9):
        kv = w12mod.KVCache.alloc(8, 1, dim, page, w12mod.KV_BF16, dev)
        kv.k.fill_(-3.0)
        kv.v.fill_(-3.0)
        x = torch.ones((len(lens) * T, 3, dim), dtype=torch.bfloat16, device=dev)
        q_out = torch.full((len(lens) * T, 1, dim), -3.0, dtype=torch.bfloat16, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        rope = _dev(w12mod.rope_table(rope_positions, 8), dev)
        w12mod.kv_append(kv, x[:, :1], x[:, 1:2], x[:, 2:], _dev(table, dev), _dev(np.array(lens, np.int32), dev), T,
                         q_out, rope, err_dev=err)
        assert int(err.item()) == w12mod.ERR_DEVICE
        wrote = (q_out[:, 0, 63] == 1.0).cpu().numpy()
        want = np.array([1, 1, 0, 0, 0, 0, 0, 0, 1, 1] if rope_positions == 64 else [0] * 8 + [1, 1], dtype=bool)
        assert np.array_equal(wrote, want)
        assert int((kv.v[:, 0, :, 0] == 1.0).sum()) == want.sum()
        assert int((kv.k[:, 0, :, 63] == 1.0).sum()) == want.sum()


@pytest.mark.parametrize("hkv,dim,page,e4m3,lens", [
    (1, 64, 16, False, [1]), (8, 128, 64, True, [1, 700, 64, 65]), (2, 128, 16, False, [33, 0, 0, 17]),
    (3, 64, 128, True, [300, 1, 127]), (5, 128, 32, True, [0, 15, 16, 1000])])
def test_read(dev, w12mod, hkv, dim, page, e4m3, lens):
    import torch
    rng = np.random.default_rng(dim + page + len(lens))
    table, n_pages = pages(rng, lens, page)
    kv = w12mod.KVCache.alloc(n_pages, hkv, dim, page, w12mod.KV_E4M3 if e4m3 else w12mod.KV_BF16, dev)
    for t in (kv.k, kv.v):
        t.copy_(_dev(rng.standard_normal(t.shape).astype(np.float32) * 40.0, dev).to(t.dtype))
    for t in (kv.k_scale, kv.v_scale):
        if t is not None:
            t.copy_(_dev(rng.random(t.shape, dtype=np.float32), dev))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    outs = [torch.empty((cu[-1], hkv, dim), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    w12mod.kv_read(kv, _dev(table, dev), _dev(cu, dev), *outs, err_dev=err)
    assert int(err.item()) == 0
    for got, values in zip(outs, cache_values(kv)):
        want = np.concatenate([request_rows(values, table, r, n, page) for r, n in enumerate(lens) if n])
        got = got.float().cpu().numpy()
        # one product of two fp32 values, rounded to fp32 and then to bf16 (exact for a bf16 cache)
        tol = (2.0 ** -8 + 2 * EPS) * np.abs(want) if e4m3 else 0.0
        assert np.all(np.abs(got - want) <= tol)


def test_read_bad_entries(dev, w12mod):
    import torch
    kv = w12mod.KVCache.alloc(2, 1, 64, 16, w12mod.KV_BF16, dev)
    kv.k.fill_(2.0)
    kv.v.fill_(2.0)
    table = torch.tensor([[0, 7], [1, -5]], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 20, 60], dtype=torch.int32, device=dev)  # request 1 is longer than its table too
    k = torch.full((60, 1, 64), 9.0, dtype=torch.bfloat16, device=dev)
    v = k.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    w12mod.kv_read(kv, table, cu, k, v, err)
    assert int(err.item()) == w12mod.ERR_DEVICE
    want = np.r_[np.full(16, 2.0), np.zeros(4), np.full(16, 2.0), np.zeros(24)]
    assert np.array_equal(k[:, 0, 3].float().cpu().numpy(), want)
    assert np.array_equal(v[:, 0, 63].float().cpu().numpy(), want)


def test_offsets_past_32_bits(dev, w12mod):
    """The last pages of a cache whose byte and element offsets pass 2^32."""
    import torch
    dim, page, hkv = 128, 128, 8
    n_pages = (1 << 32) // (dim * page * hkv) + 40  # 4.3e9 one-byte channels in each of k and v
    kv = w12mod.KVCache.alloc(n_pages, hkv, dim, page, w12mod.KV_E4M3, dev)
    T, table = 200, torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=dev)
    lens = torch.tensor([T], dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x = torch.randn(T, 24, dim, generator=g, device=dev)
    q = torch.empty((T, 8, dim), dtype=torch.bfloat16, device=dev)
    w12mod.kv_append(kv, x[:, :8], x[:, 8:16], x[:, 16:], table, lens, T, q)
    k, v = (torch.empty((T, hkv, dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
    w12mod.kv_read(kv, table, torch.tensor([0, T], dtype=torch.int32, device=dev), k, v)
    for got, want in ((k, x[:, 8:16]), (v, x[:, 16:])):
        top = want.abs().amax(-1, keepdim=True)
        tol = torch.maximum(want.abs() * (2.0 ** -4 + 2.0 ** -8), top * 2.0 ** -18) + top * 2.0 ** -20
        assert bool(((got.float() - want).abs() <= tol).all())


def test_other_stream(dev, w12mod):
    """Inputs made on a side stream and the calls on that stream: nothing is ordered by the default one."""
    import torch
    s = torch.cuda.Stream()
    kv = w12mod.KVCache.alloc(3, 2, 64, 16, w12mod.KV_BF16, dev)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = torch.randn(20, 6, 64, device=dev).to(torch.bfloat16)
        q = torch.empty((20, 2, 64), dtype=torch.bfloat16, device=dev)
        table = torch.tensor([[2, 0]], dtype=torch.int32, device=dev)
        w12mod.kv_append(kv, x[:, :2], x[:, 2:4], x[:, 4:], table, torch.tensor([20], dtype=torch.int32, device=dev),
                         20, q)
        k, v = (torch.empty((20, 2, 64), dtype=torch.bfloat16, device=dev) for _ in range(2))
        w12mod.kv_read(kv, table, torch.tensor([0, 20], dtype=torch.int32, device=dev), k, v)
    s.synchronize()
    assert torch.equal(q, x[:, :2]) and torch.equal(k, x[:, 2:4]) and torch.equal(v, x[:, 4:])
