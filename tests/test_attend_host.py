"""Argument checks of the attention call (on the CPU: every refusal comes
before a launch)."""
import ctypes
import math

import pytest

from test_kv_host import DEV, KV_REFUSALS, _kv, w12  # noqa: F401


def _attend(w12, kv=None, **kw):
    f = dict(q=DEV, qs=256, R=2, T=3, hq=4, table=DEV, blocks=4, lens=DEV, max_len=64, prefix=0, scale=0.1, out=DEV,
             os=256, lse=None, ws=DEV, wsb=1 << 30)
    f.update(kw)
    return w12.lib().w12_attend(kv or _kv(w12), f["q"], f["qs"], f["R"], f["T"], f["hq"], f["table"], f["blocks"],
                                f["lens"], f["max_len"], f["prefix"], f["scale"], f["out"], f["os"], f["lse"],
                                f["ws"], f["wsb"], None)


def test_refusals(w12):  # noqa: F811
    E = w12
    for kw, want in [(dict(q=None), E.ERR_ARG), (dict(table=None), E.ERR_ARG), (dict(lens=None), E.ERR_ARG),
                     (dict(out=None), E.ERR_ARG), (dict(scale=math.nan), E.ERR_ARG), (dict(blocks=-1), E.ERR_SHAPE),
                     (dict(R=0), E.ERR_SHAPE), (dict(R=E.ATTEND_MAX_R + 1), E.ERR_SHAPE), (dict(T=0), E.ERR_SHAPE),
                     (dict(hq=0), E.ERR_SHAPE), (dict(hq=3), E.ERR_SHAPE), (dict(max_len=-1), E.ERR_SHAPE),
                     (dict(max_len=1 << 31), E.ERR_SHAPE), (dict(prefix=-1), E.ERR_SHAPE),
                     (dict(R=512, T=1 << 22), E.ERR_SHAPE), (dict(R=512, T=4096, max_len=1 << 30), E.ERR_SHAPE),
                     (dict(q=DEV + 8), E.ERR_ALIGN), (dict(qs=260), E.ERR_ALIGN), (dict(out=DEV + 4), E.ERR_ALIGN),
                     (dict(os=258), E.ERR_ALIGN), (dict(lens=DEV + 2), E.ERR_ALIGN), (dict(lse=DEV + 2), E.ERR_ALIGN)]:
        assert _attend(w12, **kw) == want, kw
    for kw, want in KV_REFUSALS:
        assert _attend(w12, kv=_kv(w12, **kw)) == getattr(E, want), kw


def test_workspace_size_refusals(w12):  # noqa: F811
    L = w12.lib()
    assert L.w12_attend_workspace_size(None, 1, 1, 2, 10, 0) == 0
    assert L.w12_attend_workspace_size(_kv(w12), 0, 1, 2, 10, 0) == 0
    assert L.w12_attend_workspace_size(_kv(w12), 1, 1, 3, 10, 0) == 0
    assert L.w12_attend_workspace_size(_kv(w12, head_dim=80), 1, 1, 2, 10, 0) == 0


def test_binding_refusals(w12):  # noqa: F811
    import torch
    x = torch.zeros(2, 4, 64)
    for bad in (lambda: w12._heads_ptr(x, 2, 4, 64, torch.float32),        # not on a GPU
                lambda: w12._heads_ptr(x, 2, 4, 32, torch.float32),        # another shape
                lambda: w12._heads_ptr(x, 2, 4, 64, torch.bfloat16),       # another type
                lambda: w12._typed_ptr(torch.zeros(2), torch.int32, 2, "kv_len"),
                lambda: w12._typed_ptr(torch.zeros(2), torch.float32, 3, "u")):
        with pytest.raises(ValueError):
            bad()
    assert w12._typed_ptr(None, torch.float32, 3, "lse") is None
    assert ctypes.sizeof(w12._CKV) == 56
