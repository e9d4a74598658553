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


def test_fp4_checks(w12):
    import ctypes
    L = w12.lib()
    F = w12._CFP4

    def gemm(blob=DEV, K=256, N=100, scale=1.0, x=DEV, xt=1, xs=None, M=4, y=DEV, yt=0, count=1, ws=DEV, wsb=1 << 24, opt=0, no_w=False):
        arr = (F * 1)(F(blob, K, N, scale, 0))
        one = lambda p: (ctypes.c_void_p * 1)(p)  # noqa: E731
        return L.w12_fp4_gemm_batched(None if no_w else arr, one(x), xt, None if xs is None else one(xs), M, one(y), yt, count, ws,
                                      wsb, opt, None)

    assert gemm(xt=0) == gemm(xt=3) == gemm(yt=2) == gemm(opt=1) == gemm(opt=0x101) == gemm(no_w=True) == w12.ERR_ARG
    assert gemm(xs=DEV) == gemm(xt=2) == w12.ERR_ARG
    assert gemm(M=0) == gemm(M=129) == gemm(count=0) == gemm(count=9) == w12.ERR_SHAPE
    assert gemm(K=0) == gemm(K=100) == gemm(K=-128) == gemm(N=0) == gemm(N=1 << 31) == gemm(K=1 << 31) == w12.ERR_SHAPE
    assert gemm(K=1 << 24, N=1 << 24) == w12.ERR_SHAPE
    assert gemm(blob=None) == gemm(x=None) == gemm(y=None) == gemm(scale=0.0) == gemm(scale=-1.0) == w12.ERR_ARG
    assert gemm(scale=float("nan")) == gemm(scale=float("inf")) == w12.ERR_ARG
    assert gemm(blob=DEV + 128) == gemm(x=DEV + 8) == gemm(y=DEV + 2) == gemm(y=DEV + 1, yt=1) == w12.ERR_ALIGN
    assert gemm(xt=2, xs=DEV + 2) == w12.ERR_ALIGN
    assert gemm(ws=None) == w12.ERR_WORKSPACE
    assert gemm(ws=DEV + 128) == w12.ERR_ALIGN
    assert L.w12_fp4_bytes(256, 129) == 4 * 9216 and L.w12_fp4_bytes(100, 1) == L.w12_fp4_bytes(0, 1) == L.w12_fp4_bytes(128, 0) == 0
    assert L.w12_fp4_pack(None, DEV, 128, 1, DEV, None) == w12.ERR_ARG
    assert L.w12_fp4_pack(DEV, DEV, 130, 1, DEV, None) == w12.ERR_SHAPE
    assert L.w12_fp4_pack(DEV + 8, DEV, 128, 1, DEV, None) == L.w12_fp4_pack(DEV, DEV + 4, 128, 1, DEV, None) == w12.ERR_ALIGN
    assert L.w12_fp4_encode(DEV, 128, 1, 0.0, DEV, None) == L.w12_fp4_encode(None, 128, 1, 1.0, DEV, None) == w12.ERR_ARG
    assert L.w12_fp4_encode(DEV + 2, 128, 1, 1.0, DEV, None) == L.w12_fp4_encode(DEV, 128, 1, 1.0, DEV + 16, None) == w12.ERR_ALIGN
    one = F(DEV, 128, 1, 1.0, 0)
    assert L.w12_fp4_decode(ctypes.byref(one), None, None) == w12.ERR_ARG
    assert L.w12_fp4_decode(ctypes.byref(one), DEV + 4, None) == w12.ERR_ALIGN
    assert L.w12_fp4_decode(None, DEV, None) == w12.ERR_ARG


def test_verify_sampled_checks(w12):
    import ctypes
    L = w12.lib()
    C = w12._CCut

    def call(x=DEV, xt=0, q=DEV, qt=1, R=2, T=3, V=100, d=DEV, tc=None, dc=None, u=DEV, ratio=None, acc=DEV, nxt=DEV, ws=DEV, wsb=1 << 20):
        ref = lambda c: None if c is None else ctypes.byref(C(*c))  # noqa: E731
        return L.w12_verify_sampled(x, xt, q, qt, R, T, V, d, ref(tc), ref(dc), u, ratio, acc, nxt, ws, wsb, None)

    assert call(xt=2) == call(qt=2) == call(xt=-1) == w12.ERR_ARG
    assert call(R=0) == call(T=0) == call(V=0) == call(V=w12.SAMPLE_MAX_V + 1) == call(R=1 << 25, T=2) == w12.ERR_SHAPE
    assert call(x=None) == call(q=None) == call(d=None) == call(u=None) == call(acc=None) == call(nxt=None) == w12.ERR_ARG
    assert call(x=DEV + 2) == call(q=DEV + 1) == call(u=DEV + 2) == call(d=DEV + 2) == call(ratio=DEV + 1) == w12.ERR_ALIGN
    assert call(acc=DEV + 1) == call(nxt=DEV + 2) == w12.ERR_ALIGN
    assert call(tc=(DEV + 2, None, None, None)) == call(dc=(None, DEV + 1, None, None)) == w12.ERR_ALIGN
    assert call(tc=(None, None, DEV + 2, None)) == call(dc=(None, None, None, DEV + 2)) == w12.ERR_ALIGN
    assert call(ws=None) == call(wsb=256) == w12.ERR_WORKSPACE
    assert call(ws=DEV + 128) == w12.ERR_ALIGN
    assert w12.verify_sampled_workspace_size(2, 3, 100) == 256 + 512 + 256 + 256
