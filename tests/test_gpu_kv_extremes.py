"""Cache rows and lengths at the ends of their ranges."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _dev(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_largest_finite_rows_e4m3(dev, w12mod, bf16):
    """A finite row is stored however large it is; only a NaN or an infinity
    makes it NaN.  Read back, code times scale is within 3 2^-24 of the row's
    largest (whose code is 448) before it is rounded to bf16; the second channel
    is half of it, code 224, as exact."""
    import torch
    dim = 128
    tops = np.array([2.9e38, 3.05e38, 3.2e38, 3.38e38, -3.38e38, np.inf, np.nan], dtype=np.float32)
    T = len(tops)
    x = np.zeros((T, 3, dim), dtype=np.float32)
    x[:, :, 9] = tops[:, None]
    x[:, :, 70] = tops[:, None] / 2
    xd = _dev(x, dev)
    if bf16:
        xd = xd.to(torch.bfloat16)
    x = xd.float().cpu().numpy().astype(np.float64)
    kv = w12mod.KVCache.alloc(1, 1, dim, 16, w12mod.KV_E4M3, dev)
    q = torch.empty((T, 1, dim), dtype=torch.bfloat16, device=dev)
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    w12mod.kv_append(kv, xd[:, :1], xd[:, 1:2], xd[:, 2:], table, torch.tensor([T], dtype=torch.int32, device=dev), T, q)
    k, v = (torch.empty((T, 1, dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
    w12mod.kv_read(kv, table, torch.tensor([0, T], dtype=torch.int32, device=dev), k, v)
    for n, got in ((1, k), (2, v)):
        got, want = got.float().cpu().numpy().astype(np.float64)[:, 0], x[:, n]
        fine = np.isfinite(want).all(-1)
        assert fine.tolist() == [True] * 5 + [False] * 2
        assert np.all(np.abs(got[fine] - want[fine]) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want[fine]))
        assert np.all(np.isnan(got[~fine]))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_any_negative_length_is_padding(dev, w12mod, e4m3):
    """A request whose length is far below 0 has only padding tokens."""
    import torch
    T, dim = 3, 64
    lens = np.array([-1, -(1 << 31), 3 - (1 << 31), 0, 3], dtype=np.int32)
    n = len(lens) * T
    kv = w12mod.KVCache.alloc(8, 1, dim, 16, w12mod.KV_E4M3 if e4m3 else w12mod.KV_BF16, dev)
    for t in (kv.k, kv.v):
        t.view(torch.uint8).fill_(0)
    x = torch.ones((n, 3, dim), dtype=torch.bfloat16, device=dev)
    q = torch.full((n, 1, dim), -3.0, dtype=torch.bfloat16, device=dev)
    table = _dev(np.arange(len(lens), dtype=np.int32)[:, None].copy(), dev)
    rope = _dev(w12mod.rope_table(64, 8), dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    w12mod.kv_append(kv, x[:, :1], x[:, 1:2], x[:, 2:], table, _dev(lens, dev), T, q, rope, err_dev=err)
    assert int(err.item()) == 0
    assert bool((q[:-T] == -3.0).all()) and bool((q[-T:, 0, 63] == 1.0).all())
    assert int((kv.v.view(torch.uint8).flatten(1) != 0).any(-1).sum()) == 1
