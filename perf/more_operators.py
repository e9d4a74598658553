"""Measured cases of the operators around a draft model: residual addition with
root-mean-square norm (bf16 or e4m3 out), products with 4-bit weights and group
scales, and the verification of drafted tokens against the target's
probabilities.

Each case is one call of one operator on the shapes of this repository's
decoder layer (hidden size 5120, vocabulary 151936) or on generic ones.
``run`` computes it in plain torch operations in 32 bits (``own`` false) or
through the package's public calls (``own`` true).

4-bit weights (both forms): codes [N, K / 2] uint8, two e2m1 numbers a byte
(bit 3 the sign; the low four bits are the even k), scales [N, K / 16]
float8_e4m3fn, one for 16 consecutive k, and one fp32 number for the matrix.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY_ROW = 1e-30          # a row whose largest magnitude is not above this is stored as zeros
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
W_ONE = float(1 << 31)    # fixed-point one of a token's weight
U_ONE = float(1 << 24)    # of the random numbers, top_p
P_ONE = float(1 << 44)    # of a difference of probabilities

LAYER = "5120x6144,5120x1024,5120x1024,6144x5120,5120x34816,17408x5120"  # q, k, v, o, gate and up, down


# ------------------------------------------------------------------ cases

def _norm(name, **kw):
    c = dict(op="norm", n=1, dim=5120, f32=False, delta_f32=True, delta=True, e4m3=False, offset=0.0, pad=0)
    c.update(kw)
    return dict(c, name=name) if name else c


def _fp4(name, **kw):
    c = dict(op="fp4", M=1, shapes="5120x6144", e4m3=False, y_f32=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def _verify(name, **kw):
    c = dict(op="verify", R=1, T=4, V=151936, f32=True, draft_f32=True, temperature=0.8, top_k=0, top_p=1.0, min_p=0.0,
             draft_temperature=0.8, draft_top_k=0, draft_top_p=1.0)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token's hidden state between two products: the launch itself is what counts
        _norm("norm_token"),
        # draft blocks of a batch, the next product's activations in 8 bits
        _norm("norm_block_e4m3", n=128, e4m3=True),
        # a prompt of odd length, bf16 all the way, the weights stored around 0
        _norm("norm_prompt", n=8187, delta_f32=False, offset=1.0),
        # the residual stream kept in fp32 at an odd width, rows inside wider ones
        _norm("norm_odd_f32", n=3001, dim=2883, f32=True, e4m3=True, pad=5),
        # one small product: latency
        _fp4("fp4_token_small", shapes="1024x1024"),
        # a draft model's whole layer for one token: its six matrices stream once
        _fp4("fp4_layer_token", shapes=LAYER),
        # a few requests' tokens through the down projection on 8-bit activations
        _fp4("fp4_down_e4m3", M=8, shapes="17408x5120", e4m3=True, y_f32=False),
        # the largest batch through gate and up
        _fp4("fp4_gate_up_batch", M=128, shapes="5120x34816", y_f32=False),
        # a single request's short draft
        _verify("verify_one"),
        # draft blocks of 8 requests, nucleus sampling on both sides
        _verify("verify_block_top_p", R=8, T=16, f32=False, draft_f32=False, top_p=0.95, draft_top_p=0.95),
        # many requests with short drafts; the drafter picks its largest logit
        _verify("verify_batch_greedy_draft", R=32, T=5, temperature=1.0, top_k=50, draft_temperature=0.0),
        # the same number of rows at plain temperature
        _verify("verify_batch", R=16, T=8, temperature=1.0, draft_temperature=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "fp4", "fp4", "verify"])
    if op == "norm":
        dim = rng.choice([_log(rng, 60, 17000), 8 * _log(rng, 16, 2100), 128 * _log(rng, 4, 130)])
        return _norm(None, n=_log(rng, 1, min(12000, 40000000 // dim)), dim=dim, f32=rng.random() < 0.5,
                     delta_f32=rng.random() < 0.5, delta=rng.random() < 0.8, e4m3=rng.random() < 0.5,
                     offset=rng.choice([0.0, 1.0]), pad=rng.choice([0, 0, 8, 3]))
    if op == "fp4":
        M = rng.choice([1, 1, 2, 4, 8, _log(rng, 1, 128), _log(rng, 1, 128)])
        shapes = []
        for _ in range(rng.choice([1, 1, 2, 3])):
            K = 128 * _log(rng, 1, 136)
            shapes.append("%dx%d" % (K, _log(rng, 1, min(35000, 50000000 // K))))
        return _fp4(None, M=M, shapes=",".join(shapes), e4m3=rng.random() < 0.35, y_f32=rng.random() < 0.5)
    T = rng.choice([2, 3, 5, 8, 16])
    return _verify(None, R=_log(rng, 1, 128 // T), T=T, V=_log(rng, 1000, 150000), f32=rng.random() < 0.5,
                   draft_f32=rng.random() < 0.5, temperature=rng.choice([0.0, 0.6, 1.0, 1.3]),
                   top_k=rng.choice([0, 0, 20, 200]), top_p=rng.choice([1.0, 1.0, 0.9]), min_p=rng.choice([0.0, 0.0, 0.05]),
                   draft_temperature=rng.choice([0.0, 0.7, 1.0]), draft_top_k=rng.choice([0, 0, 20]),
                   draft_top_p=rng.choice([1.0, 1.0, 0.95]))


def _shapes(c):
    return [tuple(int(v) for v in s.split("x")) for s in c["shapes"].split(",")]


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _quantise_rows(y):
    """(codes, scales) of rows along the last dimension: e4m3 with scale = amax / 448."""
    amax = y.abs().amax(-1, keepdim=True)
    some = amax > TINY_ROW
    scale = torch.where(some, amax / E4M3_MAX, torch.zeros_like(amax))
    inv = torch.where(some, E4M3_MAX / amax, torch.zeros_like(amax))
    bad = ~(amax <= 3.402823466e38)
    codes = torch.where(bad, torch.zeros_like(y), (y * inv).clamp(-E4M3_MAX, E4M3_MAX))
    return codes.to(torch.float8_e4m3fn), torch.where(bad, torch.full_like(amax, math.nan), scale).squeeze(-1)


def _fp4_weights(g, K, N):
    """A trained matrix's values (normal, a few much larger), in 4 bits."""
    w = 0.02 * _randn(g, N, K)
    n = max(1, N * K // 2000)
    w.view(-1)[torch.randint(0, N * K, (n,), generator=g, device="cuda")] *= 8.0
    whole = float(w.abs().max()) / (6.0 * E4M3_MAX)
    w = w.view(N, K // 16, 16)
    scales = (w.abs().amax(-1) / (6.0 * whole)).clamp(2.0 ** -9, E4M3_MAX).to(torch.float8_e4m3fn)
    w /= scales.float()[..., None] * whole
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    codes = torch.bucketize(w.abs(), edges).to(torch.uint8) | (w < 0).to(torch.uint8) * 8
    codes = codes.view(N, K // 2, 2)
    return codes[..., 0] | codes[..., 1] * 16, scales, whole


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = case
    s = {"case": c}
    if own:
        from lossless_bit_weight_w12_gb300 import w12
    if c["op"] == "norm":
        n, dim = c["n"], c["dim"]
        kind = torch.float32 if c["f32"] else torch.bfloat16
        rows = lambda t: torch.cat([t, torch.zeros_like(t[:, :c["pad"]])], 1)[:, :dim]  # noqa: E731
        x = 2.0 * _randn(g, n, dim)
        x[:, dim // 3] *= 30.0  # a channel that is large in every token
        s["x"] = rows(x.to(kind))
        s["delta"] = rows((0.5 * _randn(g, n, dim)).to(torch.float32 if c["delta_f32"] else torch.bfloat16)) if c["delta"] else None
        s["weight"] = (1.0 - c["offset"] + 0.2 * _randn(g, dim)).to(torch.bfloat16)
        s["residual"] = torch.empty(n, dim, dtype=kind, device="cuda") if c["delta"] else None
        s["out"] = torch.empty(n, dim, dtype=torch.float8_e4m3fn if c["e4m3"] else torch.bfloat16, device="cuda")
        s["scale"] = torch.empty(n, device="cuda") if c["e4m3"] else None
        return s
    if c["op"] == "fp4":
        s["weights"], s["x"], s["x_scale"], s["y"] = [], [], [], []
        for K, N in _shapes(c):
            codes, scales, whole = _fp4_weights(g, K, N)
            s["weights"].append(w12.FP4Weight.pack(codes, scales, whole) if own else (codes, scales, whole))
            x = _randn(g, c["M"], K)
            x[:, K // 5] *= 20.0
            xs = None
            if c["e4m3"]:
                x, xs = _quantise_rows(x)
            s["x"].append(x if c["e4m3"] else x.to(torch.bfloat16))
            s["x_scale"].append(xs)
            s["y"].append(torch.empty(c["M"], N, dtype=torch.float32 if c["y_f32"] else torch.bfloat16, device="cuda"))
        if own:
            ws = w12.workspace(w12.fp4_gemm_workspace_size(s["weights"], c["M"]))
            s["batch"] = w12.FP4Batch(s["weights"], s["x"], s["y"], ws, s["x_scale"] if c["e4m3"] else None)
        return s
    R, T, V = c["R"], c["T"], c["V"]
    x = 2.0 * _randn(g, R, T, V)
    n = min(V, 24)  # the tokens that the context makes likely
    at = torch.randint(0, V, (R, T, n), generator=g, device="cuda")
    x.scatter_add_(2, at, (9.0 - 0.25 * torch.arange(n, device="cuda")).expand(R, T, n).contiguous())
    q = x[:, :T - 1] + 0.7 * _randn(g, R, T - 1, V)  # a smaller model's view of the same text
    s["logits"] = x.view(R * T, V).to(torch.float32 if c["f32"] else torch.bfloat16)
    s["draft_logits"] = q.reshape(R * (T - 1), V).to(torch.float32 if c["draft_f32"] else torch.bfloat16)
    t = c["draft_temperature"]
    z = s["draft_logits"].float()
    if t > 0:  # drawn from the drafter's probabilities: the largest logit plus noise
        z = z / t - torch.log(-torch.log(torch.rand(z.shape, generator=g, device="cuda").clamp(1e-20, 1.0 - 6e-8)))
        if c["draft_top_k"]:
            z = torch.where(s["draft_logits"].float() >= s["draft_logits"].float().topk(min(c["draft_top_k"], V))[0][:, -1:], z, -math.inf)
    s["draft"] = z.argmax(-1).to(torch.int32).view(R, T - 1)
    s["u"] = torch.rand(R, T, generator=g, device="cuda")
    f = lambda v: torch.full((R,), v, device="cuda")  # noqa: E731
    i = lambda v: torch.full((R,), v, device="cuda", dtype=torch.int32) if v else None  # noqa: E731
    s["target_cut"] = dict(temperature=f(c["temperature"]), top_k=i(c["top_k"]),
                           top_p=f(c["top_p"]) if c["top_p"] < 1.0 else None, min_p=f(c["min_p"]) if c["min_p"] > 0.0 else None)
    s["draft_cut"] = dict(temperature=f(c["draft_temperature"]), top_k=i(c["draft_top_k"]),
                          top_p=f(c["draft_top_p"]) if c["draft_top_p"] < 1.0 else None, min_p=None)
    s["out"] = {"ratio": torch.empty(R, T - 1, device="cuda"),
                "accept": torch.empty(R, dtype=torch.int32, device="cuda"),
                "next": torch.empty(R, dtype=torch.int32, device="cuda")}
    if own:
        s["ws"] = w12.workspace(w12.verify_sampled_workspace_size(R, T, V))
        s["target_cut"], s["draft_cut"] = w12.Cut(**s["target_cut"]), w12.Cut(**s["draft_cut"])
    return s


# ------------------------------------------------------------ plain forms

def _norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    if s["delta"] is not None:
        h = h + s["delta"].float()
    y = h * (1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6)) * (s["weight"].float() + c["offset"])
    out = {"residual": h.to(s["x"].dtype)} if s["delta"] is not None else {}
    if c["e4m3"]:
        out["out"], out["scale"] = _quantise_rows(y)
    else:
        out["out"] = y.to(torch.bfloat16)
    return out


def _fp4_values(codes, scales):
    """The weights but for the matrix's own number, in 32 bits: [N, K]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    N, K = codes.shape[0], 2 * codes.shape[1]
    v = table[torch.stack([codes & 15, codes >> 4], -1).long()].view(N, K // 16, 16)
    return (v * scales.float()[..., None]).view(N, K)


def _fp4_plain(s):
    out = []
    for (codes, scales, whole), x, xs, y in zip(s["weights"], s["x"], s["x_scale"], s["y"]):
        z = (x.float() @ _fp4_values(codes, scales).T) * whole
        out.append((z if xs is None else z * xs[:, None]).to(y.dtype))
    return out


def _kept(logits, n, cut):
    """Fixed-point weights [rows, V] of the tokens that the cuts keep (0 for the others)."""
    each = lambda x: x.repeat_interleave(n)[:, None]  # noqa: E731
    x = logits.float()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    mx = x.amax(-1, keepdim=True)
    t = each(cut["temperature"])
    d = torch.where(x == mx, torch.zeros_like(x), x - mx) * torch.where(t > 0, 1.0 / t, torch.ones_like(t))
    w = torch.round(torch.exp(d) * W_ONE).long()
    w = torch.where(x == -math.inf, torch.zeros_like(w), w)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices  # ties: the lowest index first
    ws = w.gather(1, order)
    rank = torch.arange(x.shape[1], device="cuda")
    keep = (rank < 1) | (t > 0).expand(-1, x.shape[1])
    if cut["top_k"] is not None:
        k = each(cut["top_k"])
        keep &= (rank < k) | (k <= 0)
    ws = torch.where(keep, ws, torch.zeros_like(ws))
    if cut["top_p"] is not None:
        p = torch.round(each(cut["top_p"]) * U_ONE).long()
        total = ws.sum(-1, keepdim=True)
        lim = p * (total >> 24) + ((p * (total & 0xFFFFFF) + 0xFFFFFF) >> 24)  # ceil(top_p * total)
        keep &= ((ws.cumsum(-1) - ws) < lim) | (rank < 1) | (p >= U_ONE)
    if cut["min_p"] is not None:
        keep &= ws >= torch.ceil(each(cut["min_p"]) * W_ONE).long()
    return torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, torch.zeros_like(ws)))


def _share(w):
    """Probabilities of whole-number weights."""
    total = w.sum(-1, keepdim=True)
    return w.float() * torch.where(total > 0, 1.0 / total.float(), torch.zeros_like(total, dtype=torch.float32))


def _verify_plain(s):
    c = s["case"]
    R, T, V = c["R"], c["T"], c["V"]
    wp = _kept(s["logits"], T, s["target_cut"]).view(R, T, V)
    p = _share(wp)
    q = _share(_kept(s["draft_logits"], T - 1, s["draft_cut"])).view(R, T - 1, V)
    d = s["draft"].long()
    there = (d >= 0) & (d < V)
    at = torch.where(there, d, torch.zeros_like(d))[..., None]
    pd = torch.where(there, p[:, :T - 1].gather(2, at)[..., 0], torch.zeros_like(s["u"][:, 1:]))
    qd = torch.where(there, q.gather(2, at)[..., 0], torch.zeros_like(pd))
    ratio = torch.where(pd >= qd, (pd > 0).float(), pd / qd)
    n = (s["u"][:, :T - 1] * qd < pd).int().cumprod(-1).sum(-1)
    # the next token: from what the target has above the draft, or after the last from the target
    r = torch.arange(R, device="cuda")
    i = n.clamp(max=T - 2)
    less = torch.where(((n < T - 1) & there[r, i])[:, None], q[r, i], torch.zeros_like(q[r, i]))
    rest = torch.round((p[r, n] - less).clamp(min=0.0) * P_ONE).long()
    whole = ((n == T - 1) | ~there[r, i])[:, None] | (rest.sum(-1, keepdim=True) == 0)
    cum = torch.where(whole, wp[r, n], rest).cumsum(-1)
    total = cum[:, -1:]
    u = torch.floor(s["u"][:, T - 1:] * U_ONE).clamp(0, U_ONE - 1).long()
    target = u * (total >> 24) + ((u * (total & 0xFFFFFF)) >> 24)  # floor(u * total)
    tok = (cum > target).int().argmax(-1)
    return {"ratio": ratio, "accept": n.int(), "next": torch.where(total[:, 0] > 0, tok, torch.full_like(tok, -1)).int()}


# ------------------------------------------------------------------- run

def run(state):
    s, c = state, state["case"]
    if own:
        from lossless_bit_weight_w12_gb300 import w12
    if c["op"] == "norm":
        if not own:
            return _norm_plain(s)
        w12.add_norm(s["x"], s["weight"], s["out"], delta=s["delta"], residual_out=s["residual"], eps=1e-6,
                     offset=c["offset"], scale_out=s["scale"])
        return {n: s[n] for n in ("residual", "out", "scale") if s[n] is not None}
    if c["op"] == "fp4":
        if not own:
            return _fp4_plain(s)
        s["batch"]()
        return list(s["y"])
    if not own:
        return _verify_plain(s)
    o = s["out"]
    w12.verify_sampled(s["logits"], s["draft_logits"], c["R"], c["T"], s["draft"], s["u"], o["accept"], o["next"],
                       s["ws"], target_cut=s["target_cut"], draft_cut=s["draft_cut"], ratio_dev=o["ratio"])
    return dict(o)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "norm":
        one = (4 if c["f32"] else 2) * (2 if c["delta"] else 1) + ((4 if c["delta_f32"] else 2) if c["delta"] else 0)
        return {"bytes": c["n"] * c["dim"] * (one + (1 if c["e4m3"] else 2)) + (4 * c["n"] if c["e4m3"] else 0) + 2 * c["dim"],
                "flops": 6.0 * c["n"] * c["dim"]}
    if c["op"] == "fp4":
        M = c["M"]
        return {"bytes": sum(K * N * 0.5625 + M * K * (1 if c["e4m3"] else 2) + M * N * (4 if c["y_f32"] else 2) for K, N in _shapes(c)),
                "flops": sum(2.0 * M * K * N for K, N in _shapes(c))}
    R, T, V = c["R"], c["T"], c["V"]
    return {"bytes": R * V * (T * (4 if c["f32"] else 2) + (T - 1) * (4 if c["draft_f32"] else 2)) + 16 * R * T,
            "flops": 4.0 * R * (2 * T - 1) * V}


# ----------------------------------------------------------------- exact

def exact(case, seed):
    """The same results from the definitions, in 64 bits."""
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        h = s["x"].double() + (s["delta"].double() if c["delta"] else 0.0)
        y = h / torch.linalg.vector_norm(torch.cat([h / math.sqrt(c["dim"]), torch.full_like(h[:, :1], 1e-3)], 1), dim=1, keepdim=True)
        y = y * (s["weight"].double() + c["offset"])
        out = {"residual": h} if c["delta"] else {}
        if c["e4m3"]:  # the values before their rounding to e4m3
            scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / E4M3_MAX
            return {**out, "out": y / scale[:, None], "scale": scale}
        return {**out, "out": y}
    if c["op"] == "fp4":
        out = []
        for (codes, scales, whole), x, xs in zip(s["weights"], s["x"], s["x_scale"]):
            N, half = codes.shape
            w = torch.empty(N, half, 2, dtype=torch.float64, device="cuda")
            for at, nib in ((0, codes & 15), (1, codes >> 4)):
                e, m = ((nib >> 1) & 3).double(), (nib & 1).double()
                v = torch.where(e > 0, (1.0 + 0.5 * m) * torch.exp2(e - 1.0), 0.5 * m)
                w[:, :, at] = torch.where(nib >= 8, -v, v)
            w = w.view(N, -1, 16) * scales.double()[..., None] * whole
            x64 = x.double() if xs is None else x.double() * xs.double()[:, None]
            out.append(torch.einsum("mk,nk->mn", x64, w.view(N, -1)))
        return out

    R, T, V = c["R"], c["T"], c["V"]

    def probability(row, token, t, top_k, top_p, min_p):
        row = row.double()
        if t <= 0:
            return float(int((row == row.max()).int().argmax()) == token)
        p = torch.softmax(row / t, 0)
        v, order = torch.sort(p, descending=True, stable=True)
        if top_k:
            v, order = v[:top_k], order[:top_k]
        if top_p < 1.0:
            n = max(1, int((torch.cumsum(v, 0) - v < top_p * v.sum()).sum()))
            v, order = v[:n], order[:n]
        if min_p > 0.0:
            v = v * (v >= min_p * p.max())
        return float((v * (order == token)).sum() / v.sum())

    ratio = []
    for r in range(R):
        for i in range(T - 1):
            tok = int(s["draft"][r, i])
            a = probability(s["logits"][r * T + i], tok, c["temperature"], c["top_k"], c["top_p"], c["min_p"])
            b = probability(s["draft_logits"][r * (T - 1) + i], tok, c["draft_temperature"], c["draft_top_k"], c["draft_top_p"], 0.0)
            ratio.append(0.0 if a == 0.0 else min(1.0, a / b) if b > 0.0 else 1.0)
    return {"ratio": torch.tensor(ratio, dtype=torch.float64).view(R, T - 1), "accept": None, "next": None}
