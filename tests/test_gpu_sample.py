"""Sampling on the GPU against its definition.

The reference works on the sorted row in double precision.  The library's
weights are 31-bit fixed point of an fp32 exponential: each is within
2^-20 (relative) + 2^-32 (of the largest) of e^((x - max) / t), so a
cumulative weight is within 2^-20 W + V 2^-32 of the exact one.  The random
numbers are placed in the middle of the drawn token's interval, and cases
whose nucleus boundary or interval is closer than that to a decision are
told apart on the host before the draw is looked at (assert in _place).
Whole-number cases (equal logits, greedy rows) are compared exactly.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _dev(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _kept(x, t, k, p, mp):
    """(weights of the staying tokens, 0 elsewhere; margin of the closest decision) in double."""
    V = len(x)
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    w = np.where(x == x.max(), 1.0, np.exp((x - x.max()) / t))
    order = np.argsort(-x, kind="stable")
    if 0 < k < V:
        order = order[:k]
    margin = 1.0
    if p < 1.0:
        ws = w[order]
        before = np.cumsum(ws) - ws
        lim = np.round(np.float32(p) * 2.0 ** 24) / 2.0 ** 24 * ws.sum()
        margin = np.abs(before - lim).min() / ws.sum()
        n = max(1, int((before < lim).sum()))
        order = order[:n]
    if mp > 0.0:
        margin = min(margin, np.abs(w[order] - np.float32(mp)).min())
        order = order[w[order] >= np.float32(mp)]
    out = np.zeros(V)
    out[order] = w[order]
    return out, margin


def _place(rng, x, t, k, p, mp):
    """A token, a random number in the middle of its interval, its probability."""
    kept, margin = _kept(x, t, k, p, mp)
    W = kept.sum()
    eps = 2.0 ** -20 + len(x) * 2.0 ** -32 / W
    assert margin > eps, "the case sits on a decision: use another seed"
    cum = np.cumsum(kept)
    for _ in range(200):
        tok = int(np.searchsorted(cum, rng.random() * W, side="right"))
        u = np.float32((cum[tok] - 0.5 * kept[tok]) / W)
        if kept[tok] / W > 4 * eps + 2.0 ** -22:
            return tok, u, kept[tok] / W, eps
    raise AssertionError("no token wide enough: use another seed")


class Call:
    def __init__(self, w12, dev, logits, R, T, u, temperature=None, top_k=None, top_p=None, min_p=None, draft=None):
        import torch
        rows, V = logits.shape
        f = lambda a, d: None if a is None else _dev(np.asarray(a, dtype=d), dev)  # noqa: E731
        self.tokens = torch.full((rows,), -9, dtype=torch.int32, device=dev)
        self.prob = torch.full((rows,), -9.0, device=dev)
        self.accept = torch.full((R,), -9, dtype=torch.int32, device=dev)
        self.next = torch.full((R,), -9, dtype=torch.int32, device=dev)
        self.ws = w12.workspace(w12.sample_workspace_size(R, T, V), dev)
        for _ in range(2):  # the second call finds the workspace as the first left it
            w12.sample(logits, R, T, f(u, np.float32), self.tokens, self.ws, f(temperature, np.float32),
                       f(top_k, np.int32), f(top_p, np.float32), f(min_p, np.float32), self.prob,
                       f(draft, np.int32) if T > 1 else None, self.accept, self.next)
        self.tok, self.pr = self.tokens.cpu().numpy(), self.prob.cpu().numpy()


CASES = [  # R, T, V, temperatures, top_k, top_p, min_p (per request, cycled); scale of the logits
    (1, 1, 1, [1.0], None, None, None, 1.0),
    (1, 1, 2, [0.7], [1], None, None, 1.0),
    (3, 1, 7, [0.5, 1.0, 2.0], [0, 2, 9], [1.0, 0.5, 0.9], None, 1.0),
    (2, 1, 1000, None, None, None, None, 2.0),
    (4, 2, 4099, [0.8, 1.0], [50, 0, 1, 4099], [0.9, 0.3, 1.0, 0.99], [0.0, 0.05, 0.0, 0.001], 2.0),
    (1, 16, 32000, [0.6], None, [0.95], None, 3.0),
    (2, 3, 32001, [1.3], [1000, 20000], [0.999, 0.7], None, 1.0),
    (1, 1, 151936, [0.8], [40], [0.9], [0.02], 2.0),
    (3, 1, 151936, [1.0, 0.9, 2.5], None, [0.9, 0.5, 0.7], [0.0, 0.0, 0.0001], 6.0),
    (1, 2, 300007, [1.0], [5000], None, None, 1.0),
    (1, 1, 524288, [0.7], None, [0.9], None, 5.0),
]


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_sample(dev, w12mod, case, bf16):
    import torch
    R, T, V, temp, top_k, top_p, min_p, scale = CASES[case]
    rng = np.random.default_rng(1000 * case + bf16)
    x = (rng.standard_normal((R * T, V)) * scale - (30.0 if case == 3 else 0.0)).astype(np.float32)
    for row in x:
        row[rng.integers(0, V, min(V, 8))] += 5.0
    xd = _dev(x, dev)
    xd = xd.to(torch.bfloat16) if bf16 else xd
    x = xd.float().cpu().numpy()
    each = lambda a, r, d: d if a is None else a[r % len(a)]  # noqa: E731
    want = [_place(rng, x[i], each(temp, i // T, 1.0), each(top_k, i // T, 0), each(top_p, i // T, 1.0),
                   each(min_p, i // T, 0.0)) for i in range(R * T)]
    draft = rng.integers(0, V, (R, T - 1))
    toks = np.array([w[0] for w in want]).reshape(R, T)
    if T > 1:
        draft[0] = toks[0, :-1]  # the first request's drafts all agree
    full = lambda a: None if a is None else [a[r % len(a)] for r in range(R)]  # noqa: E731
    c = Call(w12mod, dev, xd, R, T, [w[1] for w in want], full(temp), full(top_k), full(top_p), full(min_p), draft)
    assert c.tok.tolist() == toks.reshape(-1).tolist()
    for got, w in zip(c.pr, want):
        assert abs(got - w[2]) <= 2 * w[3] + 2.0 ** -20 * w[2]
    for r in range(R):
        n = next((i for i in range(T - 1) if draft[r, i] != toks[r, i]), T - 1)
        assert int(c.accept[r]) == n and int(c.next[r]) == toks[r, n]


@pytest.mark.parametrize("V", [5, 4096, 151936])
def test_equal_logits_exactly(dev, w12mod, V):
    """All weights are 2^31: every cut and every draw is whole-number arithmetic."""
    import torch
    u = np.array([0.0, 0.25, 0.5, 0.999999, 1.0 - 2.0 ** -24, 0.3333333], dtype=np.float32)
    n = len(u)
    x = torch.full((n, V), -3.25, device=dev)
    one = 1 << 31
    for k, p in ((0, 1.0), (3, 1.0), (V // 2, 1.0), (0, 0.5), (0, 2.0 ** -30), (V - 1, 0.75)):
        c = Call(w12mod, dev, x, n, 1, u, [1.5] * n, [k] * n, [p] * n)
        m = k if 0 < k < V else V
        pf = int(np.round(np.float32(p) * 2.0 ** 24))
        if pf < 1 << 24:
            lim = -(-pf * m * one // (1 << 24))
            m = max(1, -(-lim // one))
        want = [(int(np.float32(a) * 2.0 ** 24) * m * one >> 24) // one for a in u]
        assert c.tok.tolist() == want, (k, p)
        assert np.all(np.abs(c.pr * m - 1) <= 2.0 ** -22)


def test_threshold_inside_ties(dev, w12mod):
    """top-k and top-p end among equal logits: the lowest indices stay."""
    import torch
    V = 20000
    x = np.full(V, -1.0, dtype=np.float32)
    x[[7, 100, 15000]] = 2.0
    x[9000:9500] = 1.0
    u = np.linspace(0, 1, 64, endpoint=False).astype(np.float32)
    xd = _dev(np.tile(x, (64, 1)), dev)
    allowed = {7, 100, 15000} | set(range(9000, 9017))
    c = Call(w12mod, dev, xd, 64, 1, u, [1.0] * 64, [20] * 64)
    assert set(c.tok.tolist()) <= allowed and {7, 100, 15000, 9000, 9016} <= set(c.tok.tolist()) | {9000, 9016}
    W = 3 + 17 * np.exp(-1.0)
    for t, p in zip(c.tok, c.pr):
        assert abs(p - (1.0 if x[t] == 2.0 else np.exp(-1.0)) / W) < 1e-6
    del torch


def test_greedy_and_odd_rows(dev, w12mod):
    import torch
    V = 3001
    rng = np.random.default_rng(5)
    x = rng.standard_normal((9, V)).astype(np.float32)
    x[0, [40, 2000]] = 9.0                 # greedy, tie: the lowest index
    x[1, 5] = np.nan                       # greedy: a NaN never wins
    x[1, 77] = 8.0
    x[2, :] = -np.inf                      # nothing to sample
    x[3, :] = np.nan
    x[4, :] = -np.inf
    x[4, 1234] = -5.0                      # one token left
    x[5, [10, 20]] = np.inf                # both take everything, half each
    x[6, :] = np.where(rng.random(V) < 0.5, np.nan, -np.inf)
    x[6, 2999] = -1e30
    x[7, :] = -0.0
    x[7, 1500:] = 0.0                      # -0 and +0 are equal
    temp = [0.0, -1.0, 1.0, 1.0, 1.0, 1.0, 1.0, np.nan, 0.0]
    u = [0.9, 0.9, 0.5, 0.5, 0.999, 0.75, 0.0, 0.5, 0.0]
    for cuts in (dict(), dict(top_k=[5] * 9, top_p=[0.9] * 9, min_p=[0.1] * 9)):
        for t in (torch.float32, torch.bfloat16):
            c = Call(w12mod, dev, _dev(x, dev).to(t), 9, 1, u, temp, **cuts)
            want = [40, 77, -1, -1, 1234, 20, 2999, 0, int(np.nanargmax(_dev(x[8], dev).to(t).float().cpu().numpy()))]
            assert c.tok.tolist() == want
            assert c.pr.tolist() == [1.0, 1.0, 0.0, 0.0, 1.0, 0.5, 1.0, 1.0, 1.0]


def test_min_p_above_one_and_u_outside(dev, w12mod):
    import torch
    x = torch.tensor([[1.0, 2.0, 2.0, 0.0]] * 4, device=dev)
    c = Call(w12mod, dev, x, 4, 1, [0.5, 1.0, -1.0, np.nan], None, None, None, [1.5, 1.0, 1.0, 1.0])
    assert c.tok.tolist() == [-1, 2, 1, 1] and c.pr.tolist() == [0.0, 0.5, 0.5, 0.5]


def test_unaligned_logits(dev, w12mod):
    """Rows and a buffer that are not 16-byte aligned."""
    import torch
    rng = np.random.default_rng(9)
    V = 5003
    for t in (torch.float32, torch.bfloat16):
        base = torch.zeros(3 * V + 1, dtype=t, device=dev)
        xd = base[1:].view(3, V)
        xd.copy_(_dev(rng.standard_normal((3, V)).astype(np.float32), dev))
        x = xd.float().cpu().numpy()
        want = [_place(rng, x[i], 1.0, 100, 1.0, 0.0) for i in range(3)]
        c = Call(w12mod, dev, xd, 3, 1, [w[1] for w in want], None, [100] * 3)
        assert c.tok.tolist() == [w[0] for w in want]


def test_frequencies(dev, w12mod):
    """20000 draws from a small row follow its probabilities (chi-square, 15 degrees: below 50)."""
    import torch
    rng = np.random.default_rng(2)
    n, V = 20000, 16
    x = rng.standard_normal(V).astype(np.float32)
    c = Call(w12mod, dev, _dev(np.tile(x, (n, 1)), dev), n, 1, rng.random(n, dtype=np.float32), [0.9] * n)
    p = np.exp((x - x.max()) / 0.9)
    p /= p.sum()
    seen = np.bincount(c.tok, minlength=V)
    assert ((seen - n * p) ** 2 / (n * p)).sum() < 50
    assert isinstance(c.tokens, torch.Tensor)


def test_agrees_with_greedy_verify(dev, w12mod, oracle):
    """Temperature 0 commits what w12_verify_greedy commits."""
    from lossless_bit_weight_w12_gb300 import synth
    R, T, V = 4, 8, 32000
    rng = synth.streams(77, 2)
    lg = synth.logits(rng[0], R * T, V)
    draft = synth.draft_tokens(rng[1], oracle.argmax(lg).reshape(R, T), R, T, V)
    want = oracle.verify_greedy(lg, R, T, draft)
    c = Call(w12mod, dev, _dev(lg, dev), R, T, np.zeros(R * T), [0.0] * R, [7] * R, [0.5] * R, None, draft)
    assert c.accept.cpu().numpy().tolist() == want[0].tolist()
    assert c.next.cpu().numpy().tolist() == want[1].tolist()


def test_side_stream_and_graph(dev, w12mod):
    """On another stream than the tensors', and captured and replayed with new
    numbers: the same tokens as by itself."""
    import torch
    R, T, V = 3, 4, 40000
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x = 3 * torch.randn(R * T, V, generator=g, device=dev)
    u = torch.rand(R * T, generator=g, device=dev)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    temp, top_p = torch.full((R,), 0.8, device=dev), torch.full((R,), 0.9, device=dev)
    draft, ws = i32(R, T - 1), w12mod.workspace(w12mod.sample_workspace_size(R, T, V), dev)
    a, b = [i32(R * T), i32(R), i32(R)], [i32(R * T), i32(R), i32(R)]

    def call(o, stream=None):
        w12mod.sample(x, R, T, u, o[0], ws, temp, None, top_p, draft_dev=draft, accept_dev=o[1], next_dev=o[2],
                      stream=stream)

    call(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(b, side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(b)
    for _ in range(3):
        u.uniform_(generator=g)
        draft.copy_(a[0].view(R, T)[:, :-1])
        call(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_many_equal_logits_around_the_nucleus(dev, w12mod):
    """Logits on a coarse grid: the nucleus ends among hundreds of equal ones, of
    which the lowest indices stay (whole-number arithmetic on the weights)."""
    import torch
    V, n = 60000, 32
    rng = np.random.default_rng(8)
    x = np.round(rng.standard_normal(V) * 8).astype(np.float32) / 8
    u = np.linspace(0, 1, n, endpoint=False).astype(np.float32)
    # the library's weights (31-bit fixed point of the fp32 exponential, which torch's on the device is)
    w = torch.exp((_dev(x, dev) - float(x.max())) * 1.0).double().cpu().numpy()
    w = np.rint(w * 2.0 ** 31).astype(np.int64)
    for p in (0.3, 0.7, 0.95):
        order = np.lexsort((np.arange(V), -x))
        pf = int(np.round(np.float32(p) * 2.0 ** 24))
        lim = -(-pf * int(w.sum()) // (1 << 24))
        before = np.cumsum(w[order]) - w[order]
        kept = np.zeros(V, dtype=np.int64)
        kept[order[before < lim]] = w[order[before < lim]]
        cum = np.cumsum(kept)
        want = [int(np.searchsorted(cum, int(np.float32(a) * 2.0 ** 24) * int(cum[-1]) >> 24, side="right")) for a in u]
        for t in (torch.float32, torch.bfloat16):
            c = Call(w12mod, dev, _dev(np.tile(x, (n, 1)), dev).to(t), n, 1, u, [1.0] * n, None, [p] * n)
            assert c.tok.tolist() == want, (p, t)
