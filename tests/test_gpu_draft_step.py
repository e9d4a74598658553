"""examples/draft_step.py: a drafter of 4-bit weights, its sampled drafts verified.

The target's and the drafter's logits of every step against a plain float64 pass
over the whole text without a cache (the drafter's with its decoded weights).
Roundings on the way: queries, keys, values, attention's output and the second
norm in bf16, 2^-8 each (as in test_gpu_decode_step.py: below 2^-6 of the row's
root mean square); the drafter's normalised tokens are e4m3 besides, twice, 2^-4 /
sqrt(3) each as a uniform error: together below 2^-3.  The outcome of a step
follows from the call's own logits (test_gpu_verify_sampled.py has the rule).
"""
import importlib.util
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
EXAMPLES = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples")


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, EXAMPLES)
    spec = importlib.util.spec_from_file_location("draft_step", os.path.join(EXAMPLES, "draft_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def models(dev, w12mod, ex):
    target = ex.Block(dev)
    return target, ex.Drafter(target)


def _plain(ex, block, mats, ids):
    """Logits of every position of a text, in float64, with matrices [N, K]."""
    import torch
    x = block.emb.cpu()[torch.as_tensor(ids)].double()
    norm = lambda z: z / torch.sqrt(z.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    h, n, half = norm(x), len(ids), ex.DIM // 2
    t = block.rope.cpu().double()[:n, None]

    def turn(z):
        c, s = t[..., :half], t[..., half:]
        return torch.cat([z[..., :half] * c - z[..., half:] * s, z[..., half:] * c + z[..., :half] * s], -1)

    heads = lambda m, k: (h @ mats[m].T).view(n, k, ex.DIM)  # noqa: E731
    g = ex.HEADS // ex.KV_HEADS
    q, k, v = turn(heads("q", ex.HEADS)), turn(heads("k", ex.KV_HEADS)).repeat_interleave(g, 1), heads("v", ex.KV_HEADS).repeat_interleave(g, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) * ex.DIM ** -0.5
    s.masked_fill_(torch.ones(n, n).triu(1).bool(), -torch.inf)
    a = torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(n, -1)
    return (norm(x + a @ mats["o"].T) @ mats["lm_head"].T).numpy()


def _off(got, want):
    return np.sqrt(((got - want) ** 2).mean(-1) / (want ** 2).mean(-1)).max()


@pytest.mark.parametrize("R,T,P", [(3, 4, 200), (2, 2, 70), (5, 7, 130)])
def test_text_of_steps(dev, w12mod, ex, models, R, T, P):
    import torch
    target, drafter = models
    mats = [{m: torch.from_numpy(b.view(np.int16)).view(torch.bfloat16).double() for m, b in target.bits.items()},
            {m: w.decode().cpu().double() for m, w in drafter.w.items()}]
    prompts = np.random.default_rng(R).integers(0, ex.VOCAB, (R, P))
    one, two = (ex.Speculator(target, drafter, prompts, T, 4 * T, temperature=0.5) for _ in range(2))
    text = [list(p) for p in prompts]
    for step in range(3):
        acc, nxt, draft = one.step()
        again = two.step(graph=False)
        assert all(np.array_equal(a, b) for a, b in zip((acc, nxt, draft), again))
        lt = one.bt["logits"].cpu().double().numpy().reshape(R, T, -1)
        ld = one.draft_logits.cpu().double().numpy()
        ratio, u = one.ratio.cpu().numpy(), one.u[1].cpu().numpy()
        for r in range(R):
            ids = text[r] + list(draft[r])
            assert _off(lt[r], _plain(ex, target, mats[0], ids)[-T:]) < 2.0 ** -6, (step, r)
            assert _off(ld[r], _plain(ex, target, mats[1], ids[:-1])[-(T - 1):]) < 2.0 ** -3, (step, r)
            stay = [u[r, i] < ratio[r, i] for i in range(T - 1)]
            assert acc[r] == (stay.index(False) if False in stay else T - 1)
            assert 0 <= nxt[r] < ex.VOCAB
            text[r] += list(draft[r, :acc[r]]) + [nxt[r]]
    one.check()
    two.check()


def test_command(dev, w12mod, ex, capsys):
    assert ex.main(["--requests", "3", "--prompt", "150", "--block", "3", "--steps", "5"]) >= 15
    assert "3 requests, blocks of 3" in capsys.readouterr().out
