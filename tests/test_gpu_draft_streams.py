"""The calls around a draft model on two streams at once, each with its own workspaces:
the same bits as one after the other."""
import numpy as np
import pytest

import draft_helpers as dh

pytestmark = pytest.mark.gpu


def _chain(w12mod, dev, seed, M, R, T, V):
    """(run, outputs) of a norm, two 4-bit products of its codes and a sampled verification."""
    import torch
    rng = np.random.default_rng(seed)
    K, shapes = 1280, [(1280, 600), (1280, 2000)]
    ws4 = []
    for k, n in shapes:
        codes, scales = dh.fp4_random(rng, k, n)
        ws4.append(w12mod.FP4Weight.pack(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev).view(torch.float8_e4m3fn), 0.01))
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(dev)
    h, hs = torch.zeros(M, K, dtype=torch.float8_e4m3fn, device=dev), torch.zeros(M, device=dev)
    ys = [torch.zeros(M, n, device=dev) for _, n in shapes]
    call = w12mod.FP4Batch(ws4, [h, h], ys, w12mod.workspace(w12mod.fp4_gemm_workspace_size(ws4, M), dev), [hs, hs])
    lt = torch.from_numpy(rng.standard_normal((R * T, V)).astype(np.float32)).to(dev)
    lq = torch.from_numpy(rng.standard_normal((R * (T - 1), V)).astype(np.float32)).to(dev)
    draft = torch.from_numpy(rng.integers(0, V, (R, T - 1)).astype(np.int32)).to(dev)
    u = torch.from_numpy(rng.random((R, T)).astype(np.float32)).to(dev)
    cut = w12mod.Cut(top_p=torch.full((R,), 0.9, device=dev), top_k=torch.arange(R, device=dev).int() * 7)
    acc, nxt = (torch.zeros(R, dtype=torch.int32, device=dev) for _ in range(2))
    ratio = torch.zeros(R, T - 1, device=dev)
    wsv = w12mod.workspace(w12mod.verify_sampled_workspace_size(R, T, V), dev)

    def run():
        w12mod.add_norm(x, None, h, scale_out=hs)
        call()
        w12mod.verify_sampled(lt, lq, R, T, draft, u, acc, nxt, wsv, cut, cut, ratio)

    return run, [h.view(torch.uint8), hs, *ys, acc, nxt, ratio]


@pytest.mark.parametrize("M", [(1, 7), (16, 40), (128, 33), (2, 128)])
def test_two_streams(dev, w12mod, M):
    import torch
    chains = [_chain(w12mod, dev, 11 + i, m, 3 + 5 * i, 4, 20000 + 13 * i) for i, m in enumerate(M)]
    want = []
    for run, out in chains:
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    streams = [torch.cuda.Stream() for _ in chains]
    for _, out in chains:
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for (run, _), s in zip(chains, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (_, out), ref in zip(chains, want):
        assert all(torch.equal(a.nan_to_num(-1.0) if a.is_floating_point() else a, b.nan_to_num(-1.0) if b.is_floating_point() else b)
                   for a, b in zip(out, ref))
