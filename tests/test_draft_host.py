"""Argument checks of the draft-model calls, on the CPU (fake device addresses,
every call returns before any device access)."""
import pytest

DEV = 0x7F0000000000


@pytest.fixture(scope="module")
def w12():
    from lossless_bit_weight_w12_gb300 import build_lib, w12 as mod
    build_lib.build()
    mod.lib()
    return mod


def test_add_norm_checks(w12):
    def call(x=DEV, xs=64, xt=0, d=DEV, ds=64, dt=1, w=DEV, wt=1, offset=0.0, eps=1e-6, rows=4, dim=64, res=DEV, rs=64,
             out=DEV, os_=64, ot=1, scale=None):
        return w12.lib().w12_add_norm(x, xs, xt, d, ds, dt, w, wt, offset, eps, rows, dim, res, rs, out, os_, ot, scale, None)

    assert call(xt=2) == call(dt=2) == call(wt=2) == call(ot=0) == call(ot=3) == w12.ERR_ARG
    assert call(eps=-1e-6) == call(eps=float("nan")) == call(eps=float("inf")) == w12.ERR_ARG
    assert call(offset=float("inf")) == call(offset=float("nan")) == w12.ERR_ARG
    assert call(rows=-1) == call(rows=1 << 31) == call(dim=0) == call(dim=w12.NORM_MAX_DIM + 1) == w12.ERR_SHAPE
    assert call(os_=63) == call(rs=63) == call(os_=-64) == w12.ERR_SHAPE
    assert call(x=None) == call(out=None) == w12.ERR_ARG
    assert call(scale=DEV) == w12.ERR_ARG             # bf16 outputs have no scales
    assert call(ot=2) == w12.ERR_ARG                  # e4m3 ones have
    assert call(x=DEV + 2) == call(d=DEV + 1) == call(w=DEV + 1) == call(res=DEV + 2) == call(out=DEV + 1) == w12.ERR_ALIGN
    assert call(ot=2, scale=DEV + 2) == w12.ERR_ALIGN
    assert call(rows=0, x=None, out=None) == w12.OK
