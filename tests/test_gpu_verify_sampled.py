"""w12_verify_sampled against the definition in float64.

A weight is within 2^-20 (relative) + 2^-32 (of the row's largest) of e^((x -
max) / t) (test_gpu_sample.py), so with W the sum in units of the largest a
cumulative weight is within e W, e = 2^-20 + V 2^-32 / W, of the exact one, and a
nucleus may end up to e W elsewhere: tokens of together at most b = 2 e + (the
largest of them) of W may stay or not; no such token is drafted or drawn.  A
probability is then off by less than p (2 e + 2^-20 + 2^-22 + 2 b) + 2^-32 / W, a
ratio by the sum of both relative errors, a cumulative sum of p - q by 2 (e_p +
e_q + b_p + b_q) + 2^-19 + V 2^-45.  Random numbers are placed away from every
decision by more than that.  Whole-number cases are exact.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _dist(x, t, k, p, mp):
    """(probabilities, W, e, b, tokens that are away from every decision) of a row in float64."""
    V = len(x)
    if not t > 0:
        out = np.zeros(V)
        out[int(np.argmax(x))] = 1.0
        return out, 1.0, 0.0, 0.0, np.ones(V, dtype=bool)
    w = np.exp((x.astype(np.float64) - x.max()) / t)
    order = np.argsort(-x, kind="stable")[:k if 0 < k < V else V]
    sure, b = np.ones(V, dtype=bool), 0.0
    if p < 1.0:
        ws = w[order]
        W, before = ws.sum(), np.cumsum(ws) - ws
        e = 2.0 ** -20 + V * 2.0 ** -32 / W
        lim = np.round(np.float32(p) * 2.0 ** 24) / 2.0 ** 24 * W
        near = np.abs(before - lim) <= e * W
        sure[order[near]] = False
        n = max(1, int((before < lim).sum()))
        b = (2 * e * W + ws[near].max(initial=0.0)) / ws[:n].sum()
        order = order[:n]
    if mp > 0.0:
        near = order[np.abs(w[order] - np.float32(mp)) <= 2.0 ** -19 * mp + 2.0 ** -31]
        sure[near] = False
        order = order[w[order] >= np.float32(mp)]
        b += w[near].sum() / w[order].sum()
    out = np.zeros(V)
    out[order] = w[order]
    W = out.sum()
    return out / W, W, 2.0 ** -20 + V * 2.0 ** -32 / W, b, sure


def _call(w12mod, dev, x, q, R, T, draft, u, target=None, drafter=None):
    import torch
    V = x.shape[-1]
    f = lambda a, d: torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=d))).to(dev)  # noqa: E731
    cut = lambda c: None if c is None else w12mod.Cut(**{n: None if v is None else f(v, np.int32 if n == "top_k" else np.float32)  # noqa: E731
                                                        for n, v in c.items()})
    ratio = torch.full((R, T - 1), -9.0, device=dev)
    acc, nxt = (torch.full((R,), -9, dtype=torch.int32, device=dev) for _ in range(2))
    ws = w12mod.workspace(w12mod.verify_sampled_workspace_size(R, T, V), dev)
    ct, cd = cut(target), cut(drafter)
    for _ in range(2):
        w12mod.verify_sampled(x, q, R, T, f(draft, np.int32) if T > 1 else None, f(u, np.float32), acc, nxt, ws, ct, cd,
                              ratio if T > 1 else None)
    return acc.cpu().numpy(), nxt.cpu().numpy(), ratio.cpu().numpy()


CASES = [  # R, T, V, target (t, k, p, min_p), drafter (t, k, p, min_p): per request, cycled
    (1, 2, 5, [(1.0, 0, 1.0, 0.0)], [(1.0, 0, 1.0, 0.0)]),
    (3, 3, 1001, [(0.8, 0, 1.0, 0.0), (1.2, 0, 1.0, 0.0)], [(0.7, 0, 1.0, 0.0)]),
    (2, 5, 4099, [(1.0, 40, 0.9, 0.0), (0.6, 0, 0.8, 0.02)], [(1.0, 20, 1.0, 0.0), (0.0, 0, 1.0, 0.0)]),
    (4, 4, 32001, [(0.0, 0, 1.0, 0.0), (1.3, 0, 0.95, 0.0), (1.0, 2000, 1.0, 0.0), (1.0, 0, 1.0, 0.01)],
     [(1.0, 0, 1.0, 0.0), (0.9, 0, 0.95, 0.0), (1.0, 50, 1.0, 0.0), (0.5, 0, 1.0, 0.05)]),
    (2, 16, 151936, [(0.8, 0, 0.95, 0.0)], [(0.8, 0, 0.9, 0.0)]),
    (1, 3, 524288, [(1.0, 0, 1.0, 0.0)], [(1.0, 1, 1.0, 0.0)]),
]


@pytest.mark.parametrize("types", [(False, False), (True, False), (True, True)], ids=["f32", "bf16_f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_verify(dev, w12mod, case, types):
    import torch
    R, T, V, target, drafter = CASES[case]
    rng = np.random.default_rng(100 * case + types[0] + 2 * types[1])
    x = (2.0 * rng.standard_normal((R * T, V))).astype(np.float32)
    for row in x:
        row[rng.integers(0, V, min(V, 12))] += 6.0
    q = (x.reshape(R, T, V)[:, :-1] + 0.8 * rng.standard_normal((R, T - 1, V))).astype(np.float32).reshape(-1, V)
    xd, qd = torch.from_numpy(x).to(dev), torch.from_numpy(q).to(dev)
    xd, qd = xd.to(torch.bfloat16) if types[0] else xd, qd.to(torch.bfloat16) if types[1] else qd
    x, q = xd.float().cpu().numpy(), qd.float().cpu().numpy()
    draft, u = np.zeros((R, T - 1), dtype=np.int64), np.zeros((R, T), dtype=np.float32)
    want_acc, want_next, want_ratio, tol = [], [], np.zeros((R, T - 1)), np.zeros((R, T - 1))
    for r in range(R):
        ct, cd = target[r % len(target)], drafter[r % len(drafter)]
        stop = int(rng.integers(0, T))  # where the block is to end, if a draft can be refused there
        n = None
        for i in range(T - 1):
            p, Wp, ep, bp, sp = _dist(x[r * T + i], *ct)
            d, Wd, eq, bq, sq = _dist(q[r * (T - 1) + i], *cd)
            like = d * sp * sq
            tok = int(rng.choice(V, p=like / like.sum()))
            if i == stop:  # a token that the drafter likes more than the target, if there is one
                tok = int(np.argmax((d - p) * sp * sq))
            a, b = p[tok], d[tok]
            draft[r, i] = tok
            ratio = 0.0 if a == 0 else min(1.0, a / b)
            want_ratio[r, i] = ratio
            tol[r, i] = 0.0 if a == 0 else ratio * (
                2 * (ep + eq + bp + bq) + 2.0 ** -18 + 2.0 ** -32 / (a * Wp) + 2.0 ** -32 / (b * Wd))
            if n is not None:
                u[r, i] = rng.random()
            elif (i == stop and ratio < 0.9) or ratio == 0.0:
                u[r, i] = 0.5 * (1.0 + ratio)
                assert u[r, i] > ratio + 2 * tol[r, i]
                n = i
            else:
                u[r, i] = 0.5 * ratio
        n = T - 1 if n is None else n
        p, Wp, ep, bp, sure = _dist(x[r * T + n], *ct)
        w, eps = p, 2 * (ep + bp)
        if n < T - 1:
            d, Wd, eq, bq, sq = _dist(q[r * (T - 1) + n], *cd)
            w, sure = np.maximum(p - d, 0.0), sure & sq
            eps = 2 * (ep + eq + bp + bq) + 2.0 ** -19 + V * 2.0 ** -45
            if w.sum() == 0.0:  # p and q are one: the target's own
                w = p
        cum = np.cumsum(w)
        for _ in range(500):
            tok = int(np.searchsorted(cum, rng.random() * cum[-1], side="right"))
            if sure[tok] and w[tok] > 4 * (eps + 2.0 ** -23):
                break
        else:
            raise AssertionError("no token wide enough: use another seed")
        u[r, T - 1] = (cum[tok] - 0.5 * w[tok]) / cum[-1]
        want_acc.append(n)
        want_next.append(tok)
    each = lambda c, j, off: None if all(v[j] == off for v in c) else [c[r % len(c)][j] for r in range(R)]  # noqa: E731
    cuts = [dict(temperature=each(c, 0, 1.0), top_k=each(c, 1, 0), top_p=each(c, 2, 1.0), min_p=each(c, 3, 0.0)) for c in (target, drafter)]
    acc, nxt, ratio = _call(w12mod, dev, xd, qd, R, T, draft, u, *cuts)
    assert np.all(np.abs(ratio - want_ratio) <= tol), np.abs(ratio - want_ratio).max()
    assert acc.tolist() == want_acc
    assert nxt.tolist() == want_next


@pytest.mark.parametrize("V", [1, 2, 777, 151936])
def test_equal_logits_exactly(dev, w12mod, V):
    """p = q = 1 / V: every draft stays, the next token is floor(u V)."""
    import torch
    u = np.array([[0.999, 0.0], [0.0, 0.25], [0.5, 1.0 - 2.0 ** -24]], dtype=np.float32)
    x = torch.full((6, V), 2.5, device=dev)
    acc, nxt, ratio = _call(w12mod, dev, x, x[:3], 3, 2, [[0], [V - 1], [V // 2]], u)
    assert acc.tolist() == [1, 1, 1] and bool((ratio == 1).all())
    assert nxt.tolist() == [int(np.floor(np.float64(v) * V)) for v in u[:, 1]]


def test_rows_without_anything(dev, w12mod):
    """Masked rows, drafts that are none, drafts the target forbids, p equal to q."""
    import torch
    V, T = 300, 3
    inf = float("inf")
    x = torch.zeros(6 * T, V, device=dev)
    x[:, 7] = 50.0                       # p is token 7 but for e^-50
    q = torch.zeros(6 * (T - 1), V, device=dev)
    q[:, 7] = 50.0
    x[0 * T:1 * T] = -inf                # request 0: nothing can be sampled
    x[1 * T] = float("nan")              # 1: the first row is NaN but for one token
    x[1 * T, 9] = 1.0
    q[2 * 2] = -inf                      # 2: the drafter's row is empty
    draft = torch.full((6, T - 1), 7)
    draft[3, 0] = -1                     # 3: no draft
    draft[4, 1] = V                      # 4: one draft, then none
    draft[5, 0] = 5                      # 5: a draft that both give 0 (weights 0)
    u = np.full((6, T), 0.5, dtype=np.float32)
    acc, nxt, ratio = _call(w12mod, dev, x, q, 6, T, draft.numpy(), u)
    assert acc.tolist() == [0, 0, 2, 0, 1, 0]
    assert nxt.tolist() == [-1, 9, 7, 7, 7, 7]
    assert ratio.tolist() == [[0, 0], [0, 1], [1, 1], [0, 1], [1, 0], [0, 1]]
    # infinite logits share their row; a masked target refuses
    x = torch.zeros(2, 8, device=dev)
    x[0, 2], x[0, 5] = inf, inf
    x[1, 1] = inf
    q = torch.zeros(1, 8, device=dev)
    acc, nxt, ratio = _call(w12mod, dev, x, q, 1, 2, [[3]], [[0.0, 0.75]])
    assert acc.tolist() == [0] and ratio.tolist() == [[0.0]] and nxt.tolist() == [5]
    acc, nxt, ratio = _call(w12mod, dev, x, q, 1, 2, [[2]], [[0.9, 0.1]])
    assert acc.tolist() == [1] and ratio.tolist() == [[1.0]] and nxt.tolist() == [1]
    # min_p above 1 removes every token
    acc, nxt, _ = _call(w12mod, dev, x, q, 1, 2, [[2]], [[0.0, 0.1]], dict(min_p=[1.5]))
    assert acc.tolist() == [0] and nxt.tolist() == [-1]


@pytest.mark.parametrize("T", [1, 3])
def test_agrees_with_sample(dev, w12mod, T):
    """Where no draft is refused, the next token is the one w12_sample draws with that number."""
    import torch
    R, V = 5, 20000
    g = torch.Generator(device=dev)
    g.manual_seed(T)
    x = 3.0 * torch.randn(R * T, V, generator=g, device=dev)
    u = torch.rand(R, T, generator=g, device=dev)
    cut = dict(temperature=[0.7, 1.0, 0.0, 1.4, 0.9], top_k=[0, 30, 0, 0, 5000], top_p=[0.9, 1.0, 0.5, 0.99, 0.8])
    draft = np.full((R, T - 1), -1)
    acc, nxt, _ = _call(w12mod, dev, x, x[:R * (T - 1)] if T > 1 else None, R, T, draft, u.cpu().numpy(), cut)
    tokens = torch.empty(R, dtype=torch.int32, device=dev)
    ws = w12mod.workspace(w12mod.sample_workspace_size(R, 1, V), dev)
    f = lambda a, d: torch.tensor(a, dtype=d, device=dev)  # noqa: E731
    w12mod.sample(x.view(R, T, V)[:, 0].contiguous(), R, 1, u[:, -1].contiguous(), tokens, ws,
                  f(cut["temperature"], torch.float32), f(cut["top_k"], torch.int32), f(cut["top_p"], torch.float32))
    assert acc.tolist() == [0] * R and nxt.tolist() == tokens.tolist()


def test_tokens_are_the_targets(dev, w12mod):
    """Drafts from q, verified against p: the first committed token is distributed as p."""
    import torch
    R, V = 200000, 9
    rng = np.random.default_rng(5)
    x, q = 1.5 * rng.standard_normal(V), 1.5 * rng.standard_normal(V)
    p = np.exp(x - x.max()) / np.exp(x - x.max()).sum()
    qq = np.exp(q - q.max()) / np.exp(q - q.max()).sum()
    f = lambda a, n: torch.from_numpy(np.broadcast_to(a.astype(np.float32), (n, V)).copy()).to(dev)  # noqa: E731
    draft = rng.choice(V, size=(R, 1), p=qq)
    u = (rng.integers(0, 1 << 24, (R, 2)) / 2.0 ** 24).astype(np.float32)
    acc, nxt, _ = _call(w12mod, dev, f(x, 2 * R), f(q, R), R, 2, draft, u)
    first = np.where(acc == 1, draft[:, 0], nxt)
    got = np.bincount(first, minlength=V) / R
    assert np.all(np.abs(got - p) <= 5.0 * np.sqrt(p * (1 - p) / R)), (got, p)  # five standard deviations
    want = np.minimum(p, qq).sum()
    assert abs((acc == 1).mean() - want) <= 5.0 * np.sqrt(want * (1 - want) / R)


def test_stream_graph_and_unaligned_rows(dev, w12mod):
    import torch
    R, T, V = 3, 4, 1003  # rows on odd boundaries
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    x = 2.0 * torch.randn(R * T, V, generator=g, device=dev)
    q = (x.view(R, T, V)[:, :-1] + torch.randn(R, T - 1, V, generator=g, device=dev)).reshape(-1, V).contiguous()
    draft = q.argmax(-1).view(R, T - 1).int()
    u = torch.rand(R, T, generator=g, device=dev)
    ws = w12mod.workspace(w12mod.verify_sampled_workspace_size(R, T, V), dev)
    out = [torch.empty(R, dtype=torch.int32, device=dev) for _ in range(4)]
    ratio = torch.empty(R, T - 1, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w12mod.verify_sampled(x, q, R, T, draft, u, out[0], out[1], ws, ratio_dev=ratio)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w12mod.verify_sampled(x, q, R, T, draft, u, out[2], out[3], ws, ratio_dev=ratio)
    for _ in range(3):
        x.add_(0.3 * torch.randn(R * T, V, generator=g, device=dev))
        u.uniform_(generator=g)
        graph.replay()
        w12mod.verify_sampled(x, q, R, T, draft, u, out[0], out[1], ws)
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
        n = out[0].tolist()
        for r in range(R):  # the rule, on the call's own ratios
            stay = [float(u[r, i]) < float(ratio[r, i]) for i in range(T - 1)]
            assert n[r] == (stay.index(False) if False in stay else T - 1)


def test_refusals(dev, w12mod):
    import torch
    R, T, V = 2, 3, 64
    x, q = torch.zeros(R * T, V, device=dev), torch.zeros(R * (T - 1), V, device=dev)
    d = torch.zeros(R, T - 1, dtype=torch.int32, device=dev)
    u, ws = torch.zeros(R, T, device=dev), w12mod.workspace(w12mod.verify_sampled_workspace_size(R, T, V), dev)
    a, n = (torch.zeros(R, dtype=torch.int32, device=dev) for _ in range(2))
    call = lambda x=x, q=q, d=d, u=u, a=a, n=n, ws=ws, **k: w12mod.verify_sampled(x, q, R, T, d, u, a, n, ws, **k)  # noqa: E731
    call()
    for bad in (lambda: call(x=x.half()), lambda: call(q=q[:3]), lambda: call(q=q[:, :32]), lambda: call(d=d.long()),
                lambda: call(u=u[:1]), lambda: call(q=None), lambda: call(a=a.float()), lambda: call(x=x.t().contiguous().t()),
                lambda: call(target_cut=w12mod.Cut(temperature=torch.ones(3, device=dev))),
                lambda: call(ratio_dev=torch.zeros(3, device=dev))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(w12mod.W12Error):
        call(ws=ws[:256])
    assert w12mod.verify_sampled_workspace_size(0, 1, 5) == w12mod.verify_sampled_workspace_size(1, 1, w12mod.SAMPLE_MAX_V + 1) == 0


def _draws(w12mod, dev, x, cut, u):
    """The tokens that w12_verify_sampled and w12_sample draw from a row with each of the numbers u."""
    import torch
    n, V = len(u), len(x)
    rows = torch.from_numpy(np.broadcast_to(np.asarray(x, dtype=np.float32), (n, V)).copy()).to(dev)
    f = {k: np.full(n, v) for k, v in cut.items()}
    _, nxt, _ = _call(w12mod, dev, rows, None, n, 1, None, np.asarray(u)[:, None], f)
    tokens = torch.empty(n, dtype=torch.int32, device=dev)
    ws = w12mod.workspace(w12mod.sample_workspace_size(n, 1, V), dev)
    d = {k: torch.from_numpy(v).to(dev, torch.int32 if k == "top_k" else torch.float32) for k, v in f.items()}
    w12mod.sample(rows, n, 1, torch.from_numpy(np.asarray(u, dtype=np.float32)).to(dev), tokens, ws,
                  d.get("temperature"), d.get("top_k"), d.get("top_p"), d.get("min_p"))
    return nxt.tolist(), tokens.cpu().tolist()


U = [0.0, 2.0 ** -24, 0.25, 0.5, 0.9, 1.0 - 2.0 ** -24]


@pytest.mark.parametrize("V", [700, 20001, 151936])
@pytest.mark.parametrize("cut", [dict(top_p=0.5), dict(top_p=2.0 ** -20), dict(top_k=300), dict(top_k=500), dict(top_k=500, top_p=0.5),
                                 dict(top_k=300, top_p=0.5), dict(top_p=0.75, min_p=0.5), dict(top_p=0.75, min_p=1.25)],
                         ids=lambda c: "_".join(f"{k}{v:.2g}" for k, v in c.items()))
def test_equal_logits_under_cuts(dev, w12mod, V, cut):
    """Equal weights: the first of them stay, min(k, V) and of these ceil(p n); the
    draw is floor(u n) -- exactly, the weights being 2^31 each."""
    n = min(cut.get("top_k", V), V)
    n = int(np.ceil(cut.get("top_p", 1.0) * n))  # (p a multiple of 2^-24, so exact)
    want = [-1 if cut.get("min_p", 0.0) > 1.0 else int(float(np.float32(u)) * n) for u in U]
    got, other = _draws(w12mod, dev, np.full(V, -3.5), cut, U)
    assert got == want and other == want
    # a second, lighter kind of token among them (weight e^-1): all before it in the order
    x = np.full(V, 1.0)
    x[1::3] = 0.0
    got, other = _draws(w12mod, dev, x, cut, U)
    assert got == other


@pytest.mark.parametrize("cut", [dict(top_p=0.9), dict(top_k=50), dict(top_k=1000, top_p=0.9), dict(min_p=0.25), dict(top_k=50, top_p=0.6, min_p=0.1)],
                         ids=lambda c: "_".join(c))
@pytest.mark.parametrize("row", ["large", "hot", "flat", "cold", "tiny", "inf", "nan", "zeros", "steps", "two"])
def test_unusual_rows_under_cuts(dev, w12mod, row, cut):
    """Rows and temperatures at the ends of what there is: the same tokens as w12_sample."""
    rng = np.random.default_rng(7)
    V = 30011
    x = rng.standard_normal(V).astype(np.float32)
    t = 1.0
    if row == "large":
        x, t = x * np.float32(8e37), 3e37
    elif row == "hot":
        t = 1e30
    elif row == "flat":
        t = np.inf
        x[rng.integers(0, V, 900)] = -np.inf
    elif row == "cold":
        t = 1e-30
    elif row == "tiny":  # 1 / t is past the largest float
        x, t = x * np.float32(1e-38), 1e-40
    elif row == "inf":
        x[rng.integers(0, V, 900)] = np.inf
        x[5] = -np.inf
    elif row == "nan":
        x[rng.integers(0, V, 20000)] = np.nan
        x[rng.integers(0, V, 20000)] = -np.inf
    elif row == "zeros":  # both zeros are one logit
        x = np.where(rng.random(V) < 0.5, 0.0, -0.0).astype(np.float32)
    elif row == "steps":
        x = np.floor(4 * x) / 4
    elif row == "two":
        x[:] = -np.inf
        x[77], x[30010] = 0.0, -1.0
    got, other = _draws(w12mod, dev, x, dict(cut, temperature=t), U)
    assert got == other and min(got) >= 0


@pytest.mark.parametrize("t", [0.0, 1.0])
@pytest.mark.parametrize("qt", [0.0, 0.7])
def test_greedy_rows(dev, w12mod, t, qt):
    """Single tokens on either side, the largest more than once, or infinite."""
    import torch
    V, inf = 5000, float("inf")
    x, q = torch.zeros(8, V, device=dev), torch.zeros(4, V, device=dev)
    top = [3, 4999, 128, 2000]
    for r in range(4):
        x[2 * r, top[r]] = inf if r == 3 else 40.0
        x[2 * r + 1, 11] = 40.0
        q[r, top[r] if r else 9] = inf if r == 2 else 40.0
    x[2, 4990], x[2, 4999], q[1, 4990] = 40.0, 40.0, 40.0
    q[1, 4999] = 40.0
    # request 0: the drafter's token is another; 1: one of two equal ones; 2, 3: the same
    draft = [[9], [4990], [128], [2000]]
    one = np.full(4, 1.0, dtype=np.float32)
    acc, nxt, ratio = _call(w12mod, dev, x, q, 4, 2, draft, np.full((4, 2), 0.5), dict(temperature=t * one), dict(temperature=qt * one))
    half = t > 0 and qt == 0  # request 1: half of the target's against all of the drafter's, and u q < p fails by equality
    assert ratio[:, 0].tolist() == [0.0, 0.5 if half else 1.0, 1.0, 1.0]
    assert acc.tolist() == [0, 0 if half else 1, 1, 1] and nxt.tolist() == [3, 4999 if half else 11, 11, 11]


@pytest.mark.parametrize("R,T,V", [(700, 2, 33), (2, 300, 40), (1300, 1, 5), (9, 3, 1), (3, 2, 1027)])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_many_requests_and_long_blocks(dev, w12mod, R, T, V, bf16):
    """More requests than CTAs, more drafts than threads, rows of a few tokens on odd boundaries."""
    import torch
    rng = np.random.default_rng(R + T + V)
    dtype = torch.bfloat16 if bf16 else torch.float32
    x = torch.from_numpy(rng.standard_normal((R * T, V)).astype(np.float32)).to(dev, dtype)
    q = torch.from_numpy(rng.standard_normal((R * (T - 1), V)).astype(np.float32)).to(dev, dtype)
    draft = rng.integers(0, V, (R, T - 1))
    row = lambda z, n: [_dist(v, 1.0, 0, 1.0, 0.0) for v in z.float().cpu().numpy().reshape(n, V)]  # noqa: E731
    p, d = row(x, R * T), row(q, R * (T - 1))
    u = rng.random((R, T)).astype(np.float32)
    want, tol = np.zeros((R, T - 1)), np.zeros((R, T - 1))
    for r in range(R):
        stop = int(rng.integers(0, T))
        for i in range(T - 1):
            (pp, Wp, ep, _, _), (dd, Wd, eq, _, _) = p[r * T + i], d[r * (T - 1) + i]
            a, b = pp[draft[r, i]], dd[draft[r, i]]
            want[r, i] = ratio = min(1.0, a / b)
            tol[r, i] = ratio * (2 * (ep + eq) + 2.0 ** -18 + 2.0 ** -32 / (a * Wp) + 2.0 ** -32 / (b * Wd))
            u[r, i] = 0.5 * (1.0 + ratio) if i >= stop and ratio < 0.9 else 0.5 * ratio
    acc, nxt, ratio = _call(w12mod, dev, x, q if T > 1 else None, R, T, draft, u)
    assert np.all(np.abs(ratio - want) <= tol)
    for r in range(R):
        no = [i for i in range(T - 1) if u[r, i] > want[r, i]]
        n = no[0] if no else T - 1
        assert acc[r] == n
        w, W, e, _, _ = p[r * T + n]
        eps = 2 * e
        if n < T - 1:
            w = np.maximum(w - d[r * (T - 1) + n][0], 0.0)
            eps = 2 * (e + d[r * (T - 1) + n][2]) + 2.0 ** -19 + V * 2.0 ** -45
        cum = np.cumsum(w)
        eps = (2 * eps + 2.0 ** -23) / cum[-1]  # (of the sum so far and of the whole; u to 2^-24)
        at = np.float64(u[r, T - 1])
        assert 0 <= nxt[r] < V and w[nxt[r]] > 0
        assert (cum[nxt[r]] - w[nxt[r]]) / cum[-1] - eps <= at <= cum[nxt[r]] / cum[-1] + eps


def test_graphs_on_one_workspace(dev, w12mod):
    """Captured calls of other sizes on one workspace, replayed in turn, give what single calls give."""
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    sizes = [(2, 4, 5000), (40, 2, 301), (1, 6, 60001), (3, 1, 128)]
    ws = w12mod.workspace(max(w12mod.verify_sampled_workspace_size(*s) for s in sizes), dev)
    calls = []
    for R, T, V in sizes:
        x, q = torch.randn(R * T, V, generator=g, device=dev), torch.randn(R * (T - 1), V, generator=g, device=dev)
        u, draft = torch.rand(R, T, generator=g, device=dev), torch.randint(0, V, (R, T - 1), generator=g, device=dev, dtype=torch.int32)
        cut = w12mod.Cut(top_k=torch.full((R,), 20, dtype=torch.int32, device=dev), top_p=torch.full((R,), 0.9, device=dev))
        out = [torch.full((R,), -7, dtype=torch.int32, device=dev) for _ in range(4)]
        run = lambda a, n, w, x=x, q=q, R=R, T=T, draft=draft, u=u, cut=cut: w12mod.verify_sampled(  # noqa: E731
            x, q if T > 1 else None, R, T, draft if T > 1 else None, u, a, n, w, cut, cut)
        run(out[0], out[1], w12mod.workspace(w12mod.verify_sampled_workspace_size(R, T, V), dev))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(out[2], out[3], ws)
        calls.append((graph, out, run))  # (run holds the tensors that the graph reads)
    for _ in range(3):
        for graph, out, _ in calls:
            out[2].fill_(-8), out[3].fill_(-8)
            graph.replay()
        for _, out, _ in calls:
            assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
    assert w12mod.get_device_error(ws) == w12mod.OK


@pytest.mark.parametrize("V", [11000 * n for n in range(1, 17)] + [300001, 524288])
def test_rows_over_more_and_more_ctas(dev, w12mod, V):
    """Rows of every length that changes how many CTAs share them: the tokens that w12_sample draws."""
    import torch
    R = 40 if V > 176000 else 160
    g = torch.Generator(device=dev)
    g.manual_seed(V)
    x = 3.0 * torch.randn(R, V, generator=g, device=dev)
    u, tokens = torch.rand(R, generator=g, device=dev), torch.empty(R, dtype=torch.int32, device=dev)
    t = torch.where(torch.arange(R, device=dev) % 5 == 4, 0.0, 0.9).float()
    k = (torch.arange(R, device=dev) % 3 * 30).int()
    p = torch.where(torch.arange(R, device=dev) % 2 == 1, 0.9, 1.0).float()
    ws = w12mod.workspace(max(w12mod.sample_workspace_size(R, 1, V), w12mod.verify_sampled_workspace_size(R, 1, V)), dev)
    acc, nxt = (torch.full((R,), -5, dtype=torch.int32, device=dev) for _ in range(2))
    for cut in (dict(temperature=t), dict(temperature=t, top_k=k, top_p=p)):
        w12mod.sample(x, R, 1, u, tokens, ws, cut["temperature"], cut.get("top_k"), cut.get("top_p"))
        ws2 = w12mod.workspace(w12mod.verify_sampled_workspace_size(R, 1, V), dev)
        w12mod.verify_sampled(x, None, R, 1, None, u.view(R, 1), acc, nxt, ws2, w12mod.Cut(**cut))
        assert not bool(acc.any()) and torch.equal(nxt, tokens)
        assert w12mod.get_device_error(ws2) == w12mod.OK
