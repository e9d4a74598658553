"""The paged cache's host side: the rotary table against its formula in
double precision, and the argument checks of the cache calls (on the CPU:
every refusal comes before any CUDA call)."""
import ctypes
import math

import numpy as np
import pytest

DEV = 0x7F0000000000  # an aligned stand-in for a device address; never dereferenced


@pytest.fixture(scope="module")
def w12():
    from lossless_bit_weight_w12_gb300 import build_lib, w12 as mod
    build_lib.build()
    mod.lib()
    return mod


def _check(table, f, amp=1.0):
    """Every entry is within one rounding of the formula (2^-24 relative to 1, twice for the
    product with the amplitude in another order)."""
    p = np.arange(table.shape[0], dtype=np.float64)[:, None]
    want = np.concatenate([np.cos(p * f), np.sin(p * f)], axis=1) * amp
    # cos and sin of a large double angle: the product p f is itself rounded (2^-53 p f)
    tol = 2.0 ** -24 * amp + 2.0 ** -51 * p * f.max()
    assert np.all(np.abs(table.astype(np.float64) - want) <= tol)


@pytest.mark.parametrize("rot", [8, 24, 64, 128])
@pytest.mark.parametrize("positions", [0, 1, 777])
def test_table_plain(w12, rot, positions):
    t = w12.rope_table(positions, rot)
    assert t.shape == (positions, rot) and t.dtype == np.float32
    _check(t, 10000.0 ** (-2.0 * np.arange(rot // 2) / rot))


def test_table_long_positions(w12):
    t = w12.rope_table(200001, 16, base=500000.0)
    _check(t[[0, 131071, 200000]][:1], 500000.0 ** (-np.arange(8) / 8.0))
    p, f = 200000.0, 500000.0 ** (-np.arange(8) / 8.0)
    np.testing.assert_allclose(t[200000, :8], np.cos(p * f), atol=2.0 ** -23)
    np.testing.assert_allclose(t[200000, 8:], np.sin(p * f), atol=2.0 ** -23)


def test_table_scalings(w12):
    rot, base = 64, 10000.0
    j = np.arange(rot // 2)
    f = base ** (-2.0 * j / rot)
    _check(w12.rope_table(300, rot, base, w12.ROPE_SCALE_LINEAR, factor=4.0), f / 4.0)
    _check(w12.rope_table(300, rot, base, w12.ROPE_SCALE_BASE, factor=4.0),
           (base * 4.0 ** (rot / (rot - 2.0))) ** (-2.0 * j / rot))
    turns = 8192 * f / (2 * math.pi)
    g = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
    _check(w12.rope_table(300, rot, base, w12.ROPE_SCALE_BANDS, factor=8.0, original=8192, low=1.0, high=4.0),
           f * g + f / 8.0 * (1.0 - g))
    at = [rot * math.log(4096 / (2 * math.pi * t)) / (2 * math.log(base)) for t in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    g = 1.0 - np.clip((j - lo) / (hi - lo), 0.0, 1.0)
    fy = f * g + f / 16.0 * (1.0 - g)
    _check(w12.rope_table(300, rot, base, w12.ROPE_SCALE_YARN, factor=16.0, original=4096), fy,
           0.1 * math.log(16.0) + 1.0)
    _check(w12.rope_table(300, rot, base, w12.ROPE_SCALE_YARN, factor=16.0, original=4096, attention=1.5), fy, 1.5)


def test_table_refusals(w12):
    L = w12.lib()
    buf = np.zeros(64, dtype=np.float32)
    P = buf.ctypes.data_as(ctypes.c_void_p)

    def t(positions=1, rot=8, base=1e4, table=P, **kw):
        f = dict(mode=0, factor=1.0, original=1.0, low=1.0, high=2.0, attention=0.0)
        f.update(kw)
        sc = w12._CRopeScaling(f["mode"], 0, f["factor"], f["original"], f["low"], f["high"], f["attention"])
        return L.w12_rope_table(positions, rot, base, ctypes.byref(sc), table)

    assert t() == w12.OK
    assert L.w12_rope_table(1, 8, 1e4, None, P) == w12.OK
    assert t(positions=-1) == w12.ERR_SHAPE
    assert t(rot=0) == w12.ERR_SHAPE
    assert t(rot=12) == w12.ERR_SHAPE
    assert t(base=1.0) == w12.ERR_ARG
    assert t(base=math.nan) == w12.ERR_ARG
    assert t(table=None) == w12.ERR_ARG
    assert t(mode=5) == w12.ERR_ARG
    assert t(mode=1, factor=0.0) == w12.ERR_ARG
    assert t(mode=1, factor=math.inf) == w12.ERR_ARG
    assert t(mode=3, original=0.0) == w12.ERR_ARG
    assert t(mode=3, low=2.0, high=2.0) == w12.ERR_ARG
    assert t(mode=4, attention=-1.0) == w12.ERR_ARG


def _kv(w12, **kw):
    f = dict(k=DEV, v=DEV, ks=DEV, vs=DEV, n_pages=4, heads=2, head_dim=64, page=16, dtype=w12.KV_E4M3)
    f.update(kw)
    return ctypes.byref(w12._CKV(f["k"], f["v"], f["ks"], f["vs"], f["n_pages"], f["heads"], f["head_dim"],
                                 f["page"], f["dtype"]))


KV_REFUSALS = [(dict(dtype=2), "ERR_ARG"), (dict(heads=0), "ERR_SHAPE"), (dict(n_pages=0), "ERR_SHAPE"),
               (dict(head_dim=96), "ERR_SHAPE"), (dict(page=8), "ERR_SHAPE"), (dict(page=48), "ERR_SHAPE"),
               (dict(n_pages=1 << 26), "ERR_SHAPE"), (dict(k=None), "ERR_ARG"), (dict(v=None), "ERR_ARG"),
               (dict(ks=None), "ERR_ARG"), (dict(vs=None), "ERR_ARG"), (dict(k=DEV + 8), "ERR_ALIGN"),
               (dict(v=DEV + 4), "ERR_ALIGN"), (dict(vs=DEV + 2), "ERR_ALIGN")]


def _append(w12, kv=None, **kw):
    f = dict(q=DEV, qs=64 * 8, k=DEV, ks=64 * 8, v=DEV, vs=64 * 8, dt=w12.BF16, R=2, T=3, hq=4, table=DEV, blocks=4,
             lens=DEV, rope=DEV, positions=10, rot=64, layout=0, out=DEV, os=256, err=None)
    f.update(kw)
    return w12.lib().w12_kv_append(kv or _kv(w12), f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["dt"], f["R"],
                                   f["T"], f["hq"], f["table"], f["blocks"], f["lens"], f["rope"], f["positions"],
                                   f["rot"], f["layout"], f["out"], f["os"], f["err"], None)


def test_append_refusals(w12):
    E = w12
    assert _append(w12, R=0, q=None) == E.OK  # no request: nothing is looked at
    for kw, want in [(dict(dt=2), E.ERR_ARG), (dict(layout=2), E.ERR_ARG), (dict(R=-1), E.ERR_SHAPE),
                     (dict(T=0), E.ERR_SHAPE), (dict(hq=0), E.ERR_SHAPE), (dict(blocks=-1), E.ERR_SHAPE),
                     (dict(R=1 << 16, T=1 << 15), E.ERR_SHAPE), (dict(rot=12), E.ERR_SHAPE),
                     (dict(rot=72), E.ERR_SHAPE), (dict(positions=-1), E.ERR_SHAPE), (dict(q=None), E.ERR_ARG),
                     (dict(k=None), E.ERR_ARG), (dict(v=None), E.ERR_ARG), (dict(table=None), E.ERR_ARG),
                     (dict(lens=None), E.ERR_ARG), (dict(out=None), E.ERR_ARG), (dict(rope=None), E.ERR_ARG),
                     (dict(q=DEV + 4), E.ERR_ALIGN), (dict(dt=E.F32, k=DEV + 8), E.ERR_ALIGN),
                     (dict(out=DEV + 4), E.ERR_ALIGN), (dict(out=DEV + 8), E.ERR_ALIGN), (dict(rope=DEV + 8), E.ERR_ALIGN),
                     (dict(qs=514), E.ERR_ALIGN), (dict(os=257), E.ERR_ALIGN), (dict(err=DEV + 2), E.ERR_ALIGN)]:
        assert _append(w12, **kw) == want, kw
    for kw, want in KV_REFUSALS:
        assert _append(w12, kv=_kv(w12, **kw)) == getattr(E, want), kw
    assert w12.lib().w12_kv_append(None, DEV, 256, DEV, 256, DEV, 256, 0, 1, 1, 4, DEV, 1, DEV, None, 0, 0, 0, DEV, 256,
                                   None, None) == E.ERR_ARG


def test_read_refusals(w12):
    E = w12

    def read(kv=None, table=DEV, blocks=4, cu=DEV, R=2, tokens=10, k=DEV, v=DEV, err=None):
        return w12.lib().w12_kv_read(kv or _kv(w12), table, blocks, cu, R, tokens, k, v, err, None)

    assert read(tokens=0, table=None, k=None) == E.OK
    for kw, want in [(dict(tokens=-1), E.ERR_SHAPE), (dict(R=-1), E.ERR_SHAPE), (dict(R=0), E.ERR_SHAPE),
                     (dict(blocks=-1), E.ERR_SHAPE), (dict(table=None), E.ERR_ARG), (dict(cu=None), E.ERR_ARG),
                     (dict(k=None), E.ERR_ARG), (dict(v=None), E.ERR_ARG), (dict(k=DEV + 8), E.ERR_ALIGN),
                     (dict(cu=DEV + 1), E.ERR_ALIGN), (dict(tokens=1 << 31), E.ERR_SHAPE)]:
        assert read(**kw) == want, kw
    for kw, want in KV_REFUSALS:
        assert read(kv=_kv(w12, **kw)) == getattr(E, want), kw


def test_binding_refusals(w12):
    import torch
    bf = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w12.KVCache(bf, bf.float())
    with pytest.raises(ValueError):
        w12.KVCache(bf, bf, torch.zeros(2, 1, 16), torch.zeros(2, 1, 16))  # bf16 caches have no scales
    with pytest.raises(ValueError):
        w12.KVCache(bf.to(torch.float8_e4m3fn), bf.to(torch.float8_e4m3fn))  # e4m3 caches need them
    with pytest.raises(ValueError):
        w12.KVCache(bf, bf)  # not on a GPU
