"""One workspace for 4-bit products of all sizes, in any order, without clearing,
and one for sampled verifications: what the calls leave behind does not reach the
next one.  Tolerance of the products: test_gpu_fp4.py's."""
import numpy as np
import pytest

from test_gpu_fp4 import _check, _weight, _x

pytestmark = pytest.mark.gpu


def test_products_of_many_sizes(dev, w12mod):
    import torch
    rng = np.random.default_rng(21)
    shapes = [(128, 1), (640, 300), (5120, 257), (17408, 136), (1024, 5000), (256, 40000)]
    made = [_weight(w12mod, dev, rng, K, N, 0.01) for K, N in shapes]
    groups = [[0], [1], [2], [3], [4], [5], [1, 4], [2, 0, 1], [3, 2]]
    Ms = [1, 8, 9, 16, 17, 33, 64, 65, 128]
    need = max(w12mod.fp4_gemm_workspace_size([made[i][0] for i in g], M) for g in groups for M in Ms)
    ws = w12mod.workspace(need, dev)
    for turn in range(40):
        g, M = groups[rng.integers(len(groups))], int(rng.choice(Ms))
        e4m3 = bool(rng.integers(2))
        xs = [_x(dev, rng, M, made[i][0].K, e4m3) for i in g]
        ys = [torch.full((M, made[i][0].N), 7.0, device=dev) for i in g]
        w12mod.FP4Batch([made[i][0] for i in g], [x for x, _, _ in xs], ys, ws, [s for _, s, _ in xs] if e4m3 else None)()
        for i, (_, _, x64), y in zip(g, xs, ys):
            _check(y, x64, made[i][1], False, (turn, shapes[i], M, e4m3))
    assert w12mod.get_device_error(ws) == w12mod.OK


def test_verifications_of_many_sizes(dev, w12mod):
    import torch
    gen = torch.Generator(device=dev)
    gen.manual_seed(22)
    sizes = [(1, 1, 50), (1, 4, 151936), (3, 5, 1001), (40, 3, 4096), (8, 16, 20000), (200, 2, 777), (2, 9, 524288)]
    need = max(w12mod.verify_sampled_workspace_size(*s) for s in sizes)
    shared = w12mod.workspace(need, dev)
    order = np.random.default_rng(23).integers(0, len(sizes), 30)
    for i in order:
        R, T, V = sizes[i]
        p = 3.0 * torch.randn(R * T, V, device=dev, generator=gen)
        q = p.view(R, T, V)[:, :T - 1].reshape(-1, V) + 0.5 * torch.randn(R * (T - 1), V, device=dev, generator=gen)
        draft = torch.randint(0, V, (R, T - 1), device=dev, generator=gen, dtype=torch.int32)
        u = torch.rand(R, T, device=dev, generator=gen)
        cut = w12mod.Cut(top_p=torch.full((R,), 0.9, device=dev)) if i % 2 else None
        got = []
        for ws in (shared, w12mod.workspace(w12mod.verify_sampled_workspace_size(R, T, V), dev)):
            acc, nxt = (torch.full((R,), -7, dtype=torch.int32, device=dev) for _ in range(2))
            ratio = torch.full((R, max(T - 1, 1)), -7.0, device=dev)
            w12mod.verify_sampled(p, q if T > 1 else None, R, T, draft if T > 1 else None, u, acc, nxt, ws, cut, cut,
                                  ratio if T > 1 else None)
            got.append((acc, nxt, ratio))
        for a, b in zip(*got):
            assert torch.equal(a, b), (R, T, V)
    assert w12mod.get_device_error(shared) == w12mod.OK
