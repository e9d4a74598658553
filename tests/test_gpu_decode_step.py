"""The example of examples/decode_step.py: every step's logits against a plain
float64 pass over the whole text without a cache, tokens against the sampling
rule on the kernel's own logits.

Logits pass through bf16 roundings (embedding and norm outputs are the same
values on both sides; queries, keys, values, attention's output and the second
norm are rounded, 2^-8 each, e4m3 keys and values 2^-4): they are compared
over the whole row, root mean square, with 2^-8 sqrt(5) < 2^-6 (e4m3: the
value's rounding, uniform, is 2^-4 / sqrt(3) < 2^-4) of the row's own.
"""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def block(dev, w12mod, ex):
    return ex.Block(dev)


def _plain(ex, block, ids):
    """Logits of every position of a text, in float64."""
    import torch
    mat = lambda n: torch.from_numpy(block.bits[n].view(np.int16)).view(torch.bfloat16).double()  # noqa: E731
    x = block.emb.cpu()[torch.as_tensor(ids)]
    h = ex.norm(x).double()
    n = len(ids)
    heads = lambda m, k: (h @ mat(m).T).view(n, k, ex.DIM)  # noqa: E731
    half = ex.DIM // 2
    t = block.rope.cpu().double()[:n, None]

    def turn(z):
        c, s = t[..., :half], t[..., half:]
        a, b = z[..., :half], z[..., half:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k, v = turn(heads("q", ex.HEADS)), turn(heads("k", ex.KV_HEADS)), heads("v", ex.KV_HEADS)
    g = ex.HEADS // ex.KV_HEADS
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) * ex.DIM ** -0.5
    s.masked_fill_(torch.ones(n, n).triu(1).bool(), -torch.inf)
    a = torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(n, -1)
    y = ex.norm(x.float() + (a @ mat("o").T).float()).double()
    return (y @ mat("lm_head").T).numpy()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("R,T,P", [(3, 4, 300), (2, 8, 70), (4, 1, 150)])
def test_text_of_steps(dev, w12mod, ex, block, R, T, P, e4m3):
    rng = np.random.default_rng(R * 10 + T)
    prompt = rng.integers(0, ex.VOCAB, P)
    srv = ex.Server(block, prompt, R, T, 5 * T, e4m3, temperature=0.7)
    twin = ex.Server(block, prompt, R, T, 5 * T, e4m3, temperature=0.7)
    text = [list(prompt) for _ in range(R)]
    for step in range(4):
        draft = rng.integers(0, ex.VOCAB, (R, max(T - 1, 1))).astype(np.int32)
        import torch
        d = torch.from_numpy(draft)
        if T > 1 and step:  # a draft that comes true in part: what the same random numbers give
            state = srv.rng.get_state()
            probe = ex.Server.__new__(ex.Server)
            probe.__dict__.update(srv.__dict__)
            keep = [t.clone() for t in (srv.ids, srv.kv_len)]
            _, _, tokens = ex.Server.step(probe, d, graph=False)
            srv.ids.copy_(keep[0])
            srv.kv_len.copy_(keep[1])
            srv.rng.set_state(state)
            draft[:, 0] = tokens[:, 0]
        acc, nxt, tokens = srv.step(torch.from_numpy(draft))
        acc2, nxt2, tokens2 = twin.step(torch.from_numpy(draft), graph=False)
        assert acc.tolist() == acc2.tolist() and nxt.tolist() == nxt2.tolist() and tokens.tolist() == tokens2.tolist()
        logits = srv.b["logits"].cpu().double().numpy().reshape(R, T, -1)
        for r in range(R):
            ids = text[r] + (list(draft[r]) if T > 1 else [])
            want = _plain(ex, block, ids)[-T:]
            err = np.sqrt(((logits[r] - want) ** 2).mean(-1) / (want ** 2).mean(-1))
            assert err.max() < (2.0 ** -4 if e4m3 else 2.0 ** -6), (step, r, err)
            n = next((i for i in range(T - 1) if draft[r, i] != tokens[r, i]), T - 1)
            assert acc[r] == n and nxt[r] == tokens[r, n]
            if T > 1 and step:
                assert acc[r] >= 1
            text[r] += list(draft[r, :n]) + [nxt[r]] if T > 1 else [nxt[r]]
    srv.check()
    twin.check()


def test_command(dev, w12mod, ex, capsys):
    assert ex.main(["--requests", "3", "--prompt", "200", "--block", "4", "--steps", "6", "--e4m3"]) >= 18
    assert "3 requests under a prompt of 200" in capsys.readouterr().out
