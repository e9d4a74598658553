"""w12_fp4_*: packing, encoding and products with 4-bit weights against float64.

Tolerance of a product: x and the weights as they stand in registers are bf16
numbers, their products exact in fp32.  The tensor core adds 16 of them to an
fp32 sum at a time; if each of these 17 terms is cut at 2^-23 of the largest, one
step is off by less than 17 2^-23 S_u (S_u: the unit's sum of |x w|), the 8 steps
of a unit by 136 2^-23 S_u < 2^-15 S_u.  The up to 136 units' sums and the pieces
of a split tile are added in fp32: less than 160 2^-24 S < 2^-16 S; the
scales' products 3 roundings.  Together below 2^-14 S with S the whole sum of
|x w|; bf16 outputs add 2^-8 |y|.
"""
import numpy as np
import pytest

import draft_helpers as dh

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -14


def _weight(w12mod, dev, rng, K, N, scale):
    import torch
    codes, scales = dh.fp4_random(rng, K, N)
    w = w12mod.FP4Weight.pack(torch.from_numpy(codes).to(dev),
                              torch.from_numpy(scales).to(dev).view(torch.float8_e4m3fn), scale)
    return w, dh.fp4_values(codes, scales, scale)


def _x(dev, rng, M, K, e4m3):
    """(x, x_scale or None, float64 values)."""
    import torch
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(dev)
    if not e4m3:
        x = x.to(torch.bfloat16)
        return x, None, dh.bits_f64(x)
    c = (100.0 * x).to(torch.float8_e4m3fn)
    s = torch.from_numpy(rng.uniform(0.001, 0.02, M).astype(np.float32)).to(dev)
    return c, s, dh.bits_f64(c) * s.cpu().numpy().astype(np.float64)[:, None]


def _check(y, x64, w64, bf16, what=""):
    want, s = x64 @ w64.T, np.abs(x64) @ np.abs(w64).T
    got = dh.bits_f64(y)
    tol = TOL * s + (2.0 ** -8 * np.abs(want) if bf16 else 0.0) + 1e-30
    # (an e4m3 code past 464 is NaN: its row is NaN on both sides)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    bad = ~np.isnan(want) & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def test_decode_every_code_and_scale(dev, w12mod):
    """16 codes under every e4m3 byte, NaN and negative ones among them."""
    import torch
    nib = np.arange(16)
    codes = np.tile((nib[0::2] | nib[1::2] << 4).astype(np.uint8), (130, 16))          # K = 256
    scales = (np.arange(130 * 16) % 256).astype(np.uint8).reshape(130, 16)
    w = w12mod.FP4Weight.pack(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev).view(torch.float8_e4m3fn), 0.375)
    want = dh.fp4_values(codes, scales, 0.375)
    got = w.decode().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


@pytest.mark.parametrize("K,N,scale", [(128, 1, None), (256, 200, 0.01), (1024, 130, None), (384, 128, 1e-4)])
def test_encode(dev, w12mod, K, N, scale):
    import torch
    rng = np.random.default_rng(K + N)
    w = torch.from_numpy((0.02 * rng.standard_normal((N, K))).astype(np.float32)).to(torch.bfloat16)
    w[0, :16] = 0
    w[N // 2, 16:32] *= 1e-4
    w[N - 1, 32] = 3.0
    enc = w12mod.FP4Weight.encode(w.to(dev), scale)
    v = w.float().numpy()
    code, s = dh.fp4_encode(v, enc.scale)
    code = np.where(v < 0, code | 8, code).astype(np.uint8)
    want = dh.fp4_values(code[:, 0::2] | code[:, 1::2] << 4, s, enc.scale)
    assert np.array_equal(enc.decode().cpu().numpy(), want.astype(np.float32))
    # the same blob as packed from the plain form
    p = w12mod.FP4Weight.pack(torch.from_numpy(code[:, 0::2] | code[:, 1::2] << 4).to(dev),
                              torch.from_numpy(s).to(dev).view(torch.float8_e4m3fn), enc.scale)
    assert torch.equal(p.blob[:w12mod.lib().w12_fp4_bytes(K, N)], enc.blob[:w12mod.lib().w12_fp4_bytes(K, N)])
    if scale is None:  # the whole range is used: half a step of the largest codes (1 of 6) and of the scale
        err = np.abs(want - v).reshape(N, -1, 16)
        top = np.abs(v).reshape(N, -1, 16).max(-1, keepdims=True)
        fine = top > 64 * 2.0 ** -9 * 6 * enc.scale  # (scales far above e4m3's smallest)
        assert np.all((err <= top * (1 / 6 + 1 / 8))[np.broadcast_to(fine, err.shape)])


def test_encode_odd_values(dev, w12mod):
    import torch
    w = torch.full((2, 128), 0.5, dtype=torch.bfloat16)
    w[0, 20] = float("nan")
    w[1, 40] = float("-inf")
    got = w12mod.FP4Weight.encode(w.to(dev), 1.0).decode().cpu()
    assert bool(got[0, 16:32].isnan().all()) and not bool(got[0, :16].isnan().any()) and not bool(got[0, 32:].isnan().any())
    assert float(got[1, 40]) == -6.0 * 448.0 and not bool(got[1].isnan().any())


SHAPES = [(128, 1), (128, 128), (256, 130), (640, 300), (1024, 1024), (5120, 257), (17408, 136)]


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_gemm(dev, w12mod, M, e4m3):
    import torch
    rng = np.random.default_rng(M)
    for K, N in SHAPES:
        w, w64 = _weight(w12mod, dev, rng, K, N, 0.01)
        x, xs, x64 = _x(dev, rng, M, K, e4m3)
        ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w], M), dev)
        for dtype in (torch.float32, torch.bfloat16):
            y = torch.full((M, N), 7.0, dtype=dtype, device=dev)
            w12mod.fp4_gemm(w, x, y, ws, xs)
            _check(y, x64, w64, dtype is torch.bfloat16, (M, K, N))
            y2 = torch.full_like(y, 3.0)
            w12mod.fp4_gemm(w, x, y2, ws, xs)
            assert np.array_equal(dh.bits_f64(y), dh.bits_f64(y2), equal_nan=True)
        assert w12mod.get_device_error(ws) == w12mod.OK


@pytest.mark.parametrize("M", [1, 5, 16, 48, 128])
def test_one_hot(dev, w12mod, M):
    """A product with one weight of every column, exactly."""
    import torch
    rng = np.random.default_rng(7 * M)
    K, N = 384, 300
    w, w64 = _weight(w12mod, dev, rng, K, N, 1.0)
    ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w], M), dev)
    y = torch.empty(M, N, device=dev)
    for start in range(0, K, M):
        ks = np.arange(start, start + M) % K
        x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
        x[torch.arange(M), torch.from_numpy(ks)] = -2.0
        w12mod.fp4_gemm(w, x, y, ws)
        assert np.array_equal(y.cpu().numpy(), -2.0 * w64[:, ks].T)


@pytest.mark.parametrize("M,e4m3", [(1, False), (4, True), (16, False), (40, True), (128, False)])
def test_batched(dev, w12mod, M, e4m3):
    """A layer's products in one launch, with and without the early weight stream."""
    import torch
    rng = np.random.default_rng(M + 1)
    shapes = [(1024, 768), (1024, 128), (1024, 100), (768, 1024), (1024, 2500), (128, 5), (2432, 1024), (256, 256)]
    made = [_weight(w12mod, dev, rng, K, N, 0.02) for K, N in shapes]
    xs = [_x(dev, rng, M, K, e4m3) for K, _ in shapes]
    ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w for w, _ in made], M), dev)
    torch.cuda.synchronize()
    for options in (0, w12mod.OPT_EARLY_WEIGHTS):
        ys = [torch.empty(M, N, device=dev) for _, N in shapes]
        w12mod.FP4Batch([w for w, _ in made], [x for x, _, _ in xs], ys, ws, [s for _, s, _ in xs] if e4m3 else None, options)()
        for (w, w64), (_, _, x64), y in zip(made, xs, ys):
            _check(y, x64, w64, False, (w.K, w.N, options))
    assert w12mod.get_device_error(ws) == w12mod.OK


def test_rows_do_not_mix(dev, w12mod):
    """NaN, infinity and zero rows stay in their rows; a NaN scale in its column."""
    import torch
    rng = np.random.default_rng(11)
    K, N = 512, 260
    codes, scales = dh.fp4_random(rng, K, N)
    scales[scales == 0] = 0x30
    scales[9, 3] = 0x7F
    w = w12mod.FP4Weight.pack(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev).view(torch.float8_e4m3fn), 0.01)
    w64 = dh.fp4_values(codes, scales, 0.01)
    for M in (3, 12, 30, 70):
        x, _, x64 = _x(dev, rng, M, K, False)
        x[0, 17] = float("nan")
        x[M - 1] = 0
        x64[M - 1] = 0
        y = torch.empty(M, N, device=dev)
        ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w], M), dev)
        w12mod.fp4_gemm(w, x, y, ws)
        assert bool(y[0].isnan().all()) and bool(y[:, 9].isnan().all())
        cols = [n for n in range(N) if n != 9]
        _check(y[1:, cols], x64[1:], w64[cols], False, M)
        assert bool((y[M - 1, cols] == 0).all())


def test_stream_graph_and_shared_workspace(dev, w12mod):
    """Two captured products on one workspace, replayed on a side stream with new inputs."""
    import torch
    rng = np.random.default_rng(13)
    a, a64 = _weight(w12mod, dev, rng, 1024, 700, 0.01)
    b, b64 = _weight(w12mod, dev, rng, 640, 300, 0.01)
    x, _, _ = _x(dev, rng, 6, 1024, False)
    z, _, _ = _x(dev, rng, 20, 640, False)
    ya, yb = torch.empty(6, 700, device=dev), torch.empty(20, 300, device=dev)
    ws = w12mod.workspace(max(w12mod.fp4_gemm_workspace_size([a], 6), w12mod.fp4_gemm_workspace_size([b], 20)), dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w12mod.fp4_gemm(a, x, ya, ws)
        w12mod.fp4_gemm(b, z, yb, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w12mod.fp4_gemm(a, x, ya, ws)
        w12mod.fp4_gemm(b, z, yb, ws)
    for _ in range(3):
        x.copy_(torch.from_numpy(rng.standard_normal((6, 1024)).astype(np.float32)))
        z.copy_(torch.from_numpy(rng.standard_normal((20, 640)).astype(np.float32)))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        _check(ya, dh.bits_f64(x), a64, False)
        _check(yb, dh.bits_f64(z), b64, False)


def test_refusals(dev, w12mod):
    import torch
    rng = np.random.default_rng(17)
    w, _ = _weight(w12mod, dev, rng, 256, 64, 0.01)
    x, y = torch.zeros(2, 256, dtype=torch.bfloat16, device=dev), torch.zeros(2, 64, device=dev)
    ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w], 2), dev)
    for bad in (lambda: w12mod.fp4_gemm(w, x[:, :128], y, ws), lambda: w12mod.fp4_gemm(w, x, y[:1], ws),
                lambda: w12mod.fp4_gemm(w, x.half(), y, ws), lambda: w12mod.fp4_gemm(w, x.cpu(), y, ws),
                lambda: w12mod.FP4Weight.pack(torch.zeros(4, 64, dtype=torch.uint8, device=dev), torch.zeros(4, 8, device=dev)),
                lambda: w12mod.fp4_gemm(w, x.to(torch.float8_e4m3fn), y, ws, torch.ones(3, device=dev))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: w12mod.fp4_gemm(w, x.float(), y, ws), lambda: w12mod.fp4_gemm(w, x, y, ws[:128]),
                lambda: w12mod.fp4_gemm(w, x.to(torch.float8_e4m3fn), y, ws),
                lambda: w12mod.fp4_gemm(w, x, y, ws, torch.ones(2, device=dev)),
                lambda: w12mod.fp4_gemm(w, torch.zeros(129, 256, dtype=torch.bfloat16, device=dev), torch.zeros(129, 64, device=dev), ws),
                lambda: w12mod.FP4Weight.pack(torch.zeros(4, 32, dtype=torch.uint8, device=dev),
                                              torch.zeros(4, 4, device=dev).to(torch.float8_e4m3fn)),
                lambda: w12mod.fp4_gemm(w, x, y, ws, options=1)):
        with pytest.raises(w12mod.W12Error):
            bad()
    assert w12mod.fp4_gemm_workspace_size([w], 0) == w12mod.fp4_gemm_workspace_size([w], 129) == 0


@pytest.mark.parametrize("M,e4m3", [(3, True), (17, True), (33, False), (65, True), (128, True)])
def test_eight_matrices(dev, w12mod, M, e4m3):
    """As many matrices as a call takes, some on the same tokens, of one column to several tiles."""
    import torch
    rng = np.random.default_rng(M + 900)
    shapes = [(128, 1), (128, 513), (256, 256), (256, 31), (1280, 700), (128, 512), (256, 300), (1280, 9)]
    tokens = {K: _x(dev, rng, M, K, e4m3) for K in (128, 256, 1280)}
    pairs = [_weight(w12mod, dev, rng, K, N, 0.02) for K, N in shapes]
    xs = [tokens[K] for K, _ in shapes]
    ws = w12mod.workspace(w12mod.fp4_gemm_workspace_size([w for w, _ in pairs], M), dev)
    for options in (0, w12mod.OPT_EARLY_WEIGHTS):
        ys = [torch.full((M, N), 5.0, device=dev) for _, N in shapes]
        call = w12mod.FP4Batch([w for w, _ in pairs], [x for x, _, _ in xs], ys, ws, [s for _, s, _ in xs] if e4m3 else None, options)
        call()
        call()
        for y, (_, w64), (_, _, x64), shape in zip(ys, pairs, xs, shapes):
            _check(y, x64, w64, False, (M, shape))
    assert w12mod.get_device_error(ws) == w12mod.OK
