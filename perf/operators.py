"""Measured cases of the decode-step operators: the paged key/value cache (append
with rotary positions, read back), attention over it and sampling.

Each case is one call of one operator on the shapes of this repository's
decoder layer (48 query heads and 8 key/value heads of 128, vocabulary
151936) or on generic ones.  ``run`` computes it in plain torch operations in
32 bits (``own`` false) or through the package's public calls (``own`` true).

Cache layout (both forms): pages of ``page`` tokens, k and v
[n_pages, heads, page, head_dim] in bf16 or e4m3, and for e4m3 one fp32 scale
per token and head, [n_pages, heads, page]; ``block_table`` [R, blocks] names
the pages of each request, ``kv_len`` [R] its length with the T new tokens.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY_ROW = 1e-30          # a row whose largest magnitude is not above this is stored as zeros
W_ONE = float(1 << 31)    # fixed-point one of the sampling weights
U_ONE = float(1 << 24)    # fixed-point one of the random numbers, top_p


# ------------------------------------------------------------------ cases

def _append(name, **kw):
    c = dict(op="append", R=1, T=1, hq=48, hkv=8, dim=128, rot=128, interleaved=False, page=64,
             e4m3=False, f32=False, lo=1, hi=1)
    c.update(kw)
    return dict(c, name=name) if name else c


def _read(name, **kw):
    c = dict(op="read", R=1, hkv=8, dim=128, page=64, e4m3=False, lo=1, hi=1)
    c.update(kw)
    return dict(c, name=name) if name else c


def _attend(name, **kw):
    c = dict(op="attend", R=1, T=1, hq=48, hkv=8, dim=128, page=64, e4m3=False, prefix=0, lo=1, hi=1)
    c.update(kw)
    return dict(c, name=name) if name else c


def _sample(name, **kw):
    c = dict(op="sample", R=1, T=1, V=151936, f32=True, temperature=0.8, top_k=0, top_p=1.0, min_p=0.0)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one request enters the cache: the launch itself is what counts
        _append("append_token_bf16", lo=1500, hi=1500),
        # draft blocks of 16 tokens of 8 requests, straight from the fp32 projections, quantised
        _append("append_block_e4m3", R=8, T=16, e4m3=True, f32=True, lo=600, hi=4000),
        # two packed prompts of odd length; half of each small head rotated, neighbouring pairs
        _append("append_prompt_rot32", R=2, T=4093, hq=32, dim=64, rot=32, interleaved=True, page=32,
                e4m3=True, lo=4093, hi=8000),
        # a few short contexts are handed to a prompt pass
        _read("read_short_bf16", R=4, page=16, lo=90, hi=333),
        # the quantised contexts of a whole batch read back (moved, or given to another path)
        _read("read_batch_e4m3", R=16, e4m3=True, lo=2000, hi=14000),
        # single-token decoding of a small batch of ragged contexts: latency
        _attend("attend_token_bf16", R=4, lo=300, hi=2500),
        # one request with a very long quantised context, one token
        _attend("attend_long_e4m3", e4m3=True, lo=131000, hi=131000),
        # draft blocks of 16 tokens of 8 ragged requests on a quantised cache
        _attend("attend_block_e4m3", R=8, T=16, e4m3=True, lo=700, hi=9000),
        # 128 requests under one long system prompt (96 query rows a head and 16 requests)
        _attend("attend_prefix_bf16", R=128, prefix=16000, lo=16020, hi=16900, page=32),
        # one request's draft block, sampled: 16 rows of fp32 logits, the nucleus
        _sample("sample_block_top_p", T=16, top_p=0.95),
        # a single row: top-k, top-p and min-p together
        _sample("sample_token_all", f32=False, top_k=50, top_p=0.9, min_p=0.02),
        # the largest batch of rows, plain temperature
        _sample("sample_batch_temp", R=128, temperature=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "sample"])
    e4m3 = rng.random() < 0.5
    dim = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        R = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, 4000 // R))
        lo = _log(rng, T, T + 6000)
        return _append(None, R=R, T=T, hq=hkv * rng.choice([1, 3, 4, 6, 8]), hkv=hkv, dim=dim,
                       rot=rng.choice([dim, dim, dim // 2, 24]), interleaved=rng.random() < 0.5, page=page,
                       e4m3=e4m3, f32=rng.random() < 0.5, lo=lo, hi=lo + _log(rng, 1, 2000))
    if op == "read":
        R = _log(rng, 1, 32)
        lo = _log(rng, 1, 90000 // R)
        return _read(None, R=R, hkv=hkv, dim=dim, page=page, e4m3=e4m3, lo=lo,
                     hi=min(90000 // R, lo + _log(rng, 1, 20000)))
    if op == "attend":
        T = rng.choice([1, 1, 2, 5, 8, 16])
        R = _log(rng, 1, 128 // T)
        prefix = rng.choice([0, 0, _log(rng, 100, 12000)])
        room = max(2, (1000 if prefix else 40000 // R) - T)
        lo = prefix + T + _log(rng, 1, room)
        return _attend(None, R=R, T=T, hq=hkv * rng.choice([1, 3, 4, 6, 8]), hkv=hkv, dim=dim, page=page,
                       e4m3=e4m3, prefix=prefix, lo=lo, hi=lo + _log(rng, 1, max(2, room // 2)))
    T = rng.choice([1, 1, 4, 16])
    return _sample(None, R=_log(rng, 1, 128 // T), T=T, V=_log(rng, 1000, 150000), f32=rng.random() < 0.5,
                   temperature=rng.choice([0.0, 0.6, 1.0, 1.3]), top_k=rng.choice([0, 0, 1, 20, 200]),
                   top_p=rng.choice([1.0, 0.9, 0.98]), min_p=rng.choice([0.0, 0.05]))


def _lens(c):
    """Lengths of the R requests, spread over [lo, hi] in a mixed order."""
    R = c["R"]
    return [c["lo"] + (c["hi"] - c["lo"]) * ((i * 7) % R) // max(1, R - 1) for i in range(R)]


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pages(c, g, lens, shared=0):
    """(block_table, n_pages): pages of each request in a random order; the
    first `shared` pages of every request are the same ones."""
    page, R = c["page"], c["R"]
    need = [-(-n // page) for n in lens]
    total = shared + sum(n - shared for n in need)
    ids = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(R, max(need), dtype=torch.int32, device="cuda")
    at = shared
    for r in range(R):
        table[r, :shared] = ids[:shared]
        table[r, shared:need[r]] = ids[at:at + need[r] - shared]
        at += need[r] - shared
    return table, total + 3


def _quantise(x):
    """(codes, scales) of rows along the last dimension: e4m3 with scale = amax / 448."""
    amax = x.abs().amax(-1, keepdim=True)
    some = amax > TINY_ROW
    scale = torch.where(some, amax / E4M3_MAX, torch.zeros_like(amax))
    inv = torch.where(some, E4M3_MAX / amax, torch.zeros_like(amax))
    bad = ~(amax <= 3.0e38)
    codes = torch.where(bad, torch.zeros_like(x), (x * inv).clamp(-E4M3_MAX, E4M3_MAX))
    return codes.to(torch.float8_e4m3fn), torch.where(bad, torch.full_like(amax, math.nan), scale).squeeze(-1)


def _cache(c, g, n_pages):
    """A cache whose every page holds rows (the tail of a last page what another request left there)."""
    shape = (n_pages, c["hkv"], c["page"], c["dim"])
    s = {}
    for n in ("k", "v"):
        x = _randn(g, *shape)
        if n == "k":  # a few channels are much larger than the others
            x *= 1.0 + 3.0 * (torch.arange(c["dim"], device="cuda") % 37 == 5).float()
        if c["e4m3"]:
            s[n], s[n + "_scale"] = _quantise(x)
        else:
            s[n] = x.to(torch.bfloat16)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = case
    s = {"case": c}
    if c["op"] == "sample":
        R, T, V = c["R"], c["T"], c["V"]
        x = 2.0 * _randn(g, R * T, V)
        n = min(V, 24)  # the tokens that the context makes likely
        at = torch.randint(0, V, (R * T, n), generator=g, device="cuda")
        x.scatter_add_(1, at, (9.0 - 0.25 * torch.arange(n, device="cuda")).expand(R * T, n).contiguous())
        s["logits"] = x if c["f32"] else x.to(torch.bfloat16)
        s["u"] = torch.rand(R * T, generator=g, device="cuda")
        s["temperature"] = torch.full((R,), c["temperature"], device="cuda")
        s["top_k"] = torch.full((R,), c["top_k"], dtype=torch.int32, device="cuda") if c["top_k"] else None
        s["top_p"] = torch.full((R,), c["top_p"], device="cuda") if c["top_p"] < 1.0 else None
        s["min_p"] = torch.full((R,), c["min_p"], device="cuda") if c["min_p"] > 0.0 else None
        s["draft"] = torch.randint(0, V, (R, T - 1), generator=g, device="cuda", dtype=torch.int32) if T > 1 else None
        s["out"] = {"tokens": torch.empty(R * T, dtype=torch.int32, device="cuda"),
                    "prob": torch.empty(R * T, device="cuda"),
                    "accept": torch.empty(R, dtype=torch.int32, device="cuda"),
                    "next": torch.empty(R, dtype=torch.int32, device="cuda")}
        if own:
            from lossless_bit_weight_w12_gb300 import w12
            s["ws"] = w12.workspace(w12.sample_workspace_size(R, T, V))
        return s

    lens = _lens(c)
    shared = c.get("prefix", 0) // c["page"]
    s["block_table"], n_pages = _pages(c, g, lens, shared)
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s.update(_cache(c, g, n_pages))
    hkv, dim = c["hkv"], c["dim"]
    if c["op"] == "append":
        n, hq = c["R"] * c["T"], c["hq"]
        qkv = _randn(g, n, hq + 2 * hkv, dim)  # the projections' output, one row per token
        s["qkv"] = qkv if c["f32"] else qkv.to(torch.bfloat16)
        f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        a = torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None] * f
        s["table"] = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
        s["q_out"] = torch.empty(n, hq, dim, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "read":
        s["cu_len"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["k_out"] = torch.empty(sum(lens), hkv, dim, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        if c["prefix"] % c["page"]:  # the page that the prefix ends in: each request has its copy
            for n in [x for x in ("k", "v", "k_scale", "v_scale") if x in s]:
                last, stop = s["block_table"][:, shared].long(), c["prefix"] % c["page"]
                s[n][last, :, :stop] = s[n][last[:1], :, :stop].expand(c["R"], *s[n][last[:1], :, :stop].shape[1:])
        s["q"] = (1.5 * _randn(g, c["R"] * c["T"], c["hq"], dim)).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(c["R"] * c["T"], c["hq"], device="cuda")
    if own:
        from lossless_bit_weight_w12_gb300 import w12
        s["kv"] = w12.KVCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
        if c["op"] == "attend":
            s["ws"] = w12.workspace(w12.attend_workspace_size(s["kv"], c["R"], c["T"], c["hq"], max(lens), c["prefix"]))
            s["max_len"] = max(lens)
    return s


# ------------------------------------------------------------ plain forms

def _slots(s, pos):
    """Page and row of token `pos` [R, n] of each request."""
    page = s["case"]["page"]
    return s["block_table"].gather(1, torch.div(pos, page, rounding_mode="floor")).long(), pos % page


def _rotate(x, table, pos, c):
    """Rotary positions on the first `rot` of the head's channels, in 32 bits."""
    rot, h = c["rot"], c["rot"] // 2
    cos, sin = table[pos][:, None, :h], table[pos][:, None, h:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :h], x[..., h:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([ra, rb], -1).flatten(-2) if c["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([head, x[..., rot:]], -1)


def _append_plain(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    pos = s["kv_len"].long()[:, None] - c["T"] + torch.arange(c["T"], device="cuda")
    at, row = (x.reshape(-1) for x in _slots(s, pos))
    x = s["qkv"].float()
    turned = _rotate(x[:, :hq + hkv], s["table"], pos.reshape(-1), c)
    q, k, v = turned[:, :hq].to(torch.bfloat16), turned[:, hq:], x[:, hq + hkv:]
    for n, new in (("k", k), ("v", v)):
        if c["e4m3"]:
            codes, scale = _quantise(new)
            s[n].view(torch.uint8)[at, :, row] = codes.view(torch.uint8)
            s[n + "_scale"][at, :, row] = scale
        else:
            s[n][at, :, row] = new.to(torch.bfloat16)
    return q


def _rows(s, n, idx):
    """Cache rows of the pages `idx` [...] as values in 32 bits: [..., heads, page, dim]."""
    if s["case"]["e4m3"]:
        return s[n].view(torch.uint8)[idx].view(torch.float8_e4m3fn).float() * s[n + "_scale"][idx][..., None]
    return s[n][idx].float()


def _read_plain(s):
    total = s["k_out"].shape[0]
    t = torch.arange(total, device="cuda")
    r = torch.searchsorted(s["cu_len"][1:].contiguous(), t.to(torch.int32), right=True)
    pos = t - s["cu_len"].long()[r]
    page = s["case"]["page"]
    at, row = s["block_table"][r, torch.div(pos, page, rounding_mode="floor")].long(), pos % page
    out = []
    for n in ("k", "v"):
        x = s[n].view(torch.uint8)[at, :, row].view(torch.float8_e4m3fn).float() * s[n + "_scale"][at, :, row][..., None] \
            if s["case"]["e4m3"] else s[n][at, :, row]
        out.append(x.to(torch.bfloat16))
    return {"k": out[0], "v": out[1]}


def _attend_plain(s):
    c = s["case"]
    R, T, hkv, dim = c["R"], c["T"], c["hkv"], c["dim"]
    G = c["hq"] // hkv
    idx = s["block_table"].long()
    L = idx.shape[1] * c["page"]
    k, v = (_rows(s, n, idx).transpose(1, 2).reshape(R, hkv, L, dim) for n in ("k", "v"))
    q = s["q"].float().view(R, T, hkv, G, dim).permute(0, 2, 1, 3, 4).reshape(R, hkv, T * G, dim)
    key = torch.arange(L, device="cuda")
    pos = s["kv_len"].long()[:, None] - T + torch.arange(T, device="cuda")
    seen = (key <= pos[..., None])[:, None, :, None, :].expand(R, 1, T, G, L).reshape(R, 1, T * G, L)
    sc = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(dim))
    sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(sc - m0)
    l = p.sum(-1, keepdim=True)
    v = torch.where((key < s["kv_len"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = (p @ v) / torch.where(l == 0, torch.ones_like(l), l)
    back = lambda x: x.view(R, hkv, T, G, -1).permute(0, 2, 1, 3, 4).reshape(R * T, c["hq"], -1)  # noqa: E731
    return {"out": back(o).to(torch.bfloat16), "lse": back(m0 + torch.log(l)).squeeze(-1)}


def _sample_plain(s):
    c = s["case"]
    R, T, V = c["R"], c["T"], c["V"]
    each = lambda x: x.repeat_interleave(T)[:, None]  # noqa: E731
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    mx = x.amax(-1, keepdim=True)
    t = each(s["temperature"])
    # weights relative to the row's largest, in fixed point: their sums do not depend on the order
    d = torch.where(x == mx, torch.zeros_like(x), x - mx) * torch.where(t > 0, 1.0 / t, torch.ones_like(t))
    w = torch.round(torch.exp(d) * W_ONE).long()
    w = torch.where(x == -math.inf, torch.zeros_like(w), w)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices  # ties: the lowest index first
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")
    keep = (rank < 1) | (t > 0).expand(-1, V)
    if s["top_k"] is not None:
        k = each(s["top_k"])
        keep &= (rank < k) | (k <= 0)
    ws = torch.where(keep, ws, torch.zeros_like(ws))
    if s["top_p"] is not None:
        p = torch.round(each(s["top_p"]) * U_ONE).long()
        total = ws.sum(-1, keepdim=True)
        lim = p * (total >> 24) + ((p * (total & 0xFFFFFF) + 0xFFFFFF) >> 24)  # ceil(top_p * total)
        keep &= ((ws.cumsum(-1) - ws) < lim) | (rank < 1) | (p >= U_ONE)
    if s["min_p"] is not None:
        keep &= ws >= torch.ceil(each(s["min_p"]) * W_ONE).long()
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, torch.zeros_like(ws)))
    cum = kept.cumsum(-1)
    total = cum[:, -1:]
    u = torch.floor(s["u"] * U_ONE).clamp(0, U_ONE - 1).long()[:, None]
    target = u * (total >> 24) + ((u * (total & 0xFFFFFF)) >> 24)  # floor(u * total)
    tok = (cum > target).int().argmax(-1)
    none = total[:, 0] == 0
    prob = kept.gather(1, tok[:, None])[:, 0].float() / total[:, 0].clamp(min=1).float()
    tok = torch.where(none, torch.full_like(tok, -1), tok)
    out = {"tokens": tok.int(), "prob": prob}
    g = tok.view(R, T)
    if T > 1:
        agree = (g[:, :T - 1] == s["draft"]).int().cumprod(-1).sum(-1)
        out["accept"], out["next"] = agree.int(), g.gather(1, agree[:, None])[:, 0].int()
    return out


# ------------------------------------------------------------------- run

def run(state):
    s, c = state, state["case"]
    if own:
        from lossless_bit_weight_w12_gb300 import w12
    if c["op"] == "append":
        if own:
            hq, hkv, x = c["hq"], c["hkv"], s["qkv"]
            w12.kv_append(s["kv"], x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], s["block_table"], s["kv_len"],
                          c["T"], s["q_out"], s["table"],
                          w12.ROPE_INTERLEAVED if c["interleaved"] else w12.ROPE_HALF)
            q = s["q_out"]
        else:
            q = _append_plain(s)
        return {"q": q, **{n: s[n] for n in ("k", "v", "k_scale", "v_scale") if n in s}}
    if c["op"] == "read":
        if own:
            w12.kv_read(s["kv"], s["block_table"], s["cu_len"], s["k_out"], s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        return _read_plain(s)
    if c["op"] == "attend":
        if own:
            w12.attend(s["kv"], s["q"], s["block_table"], s["kv_len"], c["T"], s["max_len"], s["out"], s["ws"],
                       prefix_len=c["prefix"], lse_dev=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        return _attend_plain(s)
    if own:
        o, many = s["out"], c["T"] > 1
        w12.sample(s["logits"], c["R"], c["T"], s["u"], o["tokens"], s["ws"], s["temperature"], s["top_k"],
                   s["top_p"], s["min_p"], prob_dev=o["prob"], draft_dev=s["draft"],
                   accept_dev=o["accept"] if many else None, next_dev=o["next"] if many else None)
        return dict(o) if many else {"tokens": o["tokens"], "prob": o["prob"]}
    return _sample_plain(s)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "sample":
        n = c["R"] * c["T"]
        return {"bytes": n * c["V"] * (4 if c["f32"] else 2) + 16 * n, "flops": 4.0 * n * c["V"]}
    lens, hkv, dim = _lens(c), c["hkv"], c["dim"]
    row = 2 * hkv * (dim + 4 if c["e4m3"] else 2 * dim)  # a token's k and v in the cache
    if c["op"] == "append":
        n, hq = c["R"] * c["T"], c["hq"]
        return {"bytes": n * ((hq + 2 * hkv) * dim * (4 if c["f32"] else 2) + 2 * hq * dim + row + 4 * c["rot"]),
                "flops": 3.0 * n * (hq + hkv) * c["rot"] + (4.0 * n * hkv * dim if c["e4m3"] else 0.0)}
    if c["op"] == "read":
        return {"bytes": sum(lens) * (row + 4 * hkv * dim), "flops": 2.0 * sum(lens) * hkv * dim}
    n = c["R"] * c["T"]
    unique = c["prefix"] + sum(x - c["prefix"] for x in lens)
    pairs = sum(x - c["T"] + 1 + i for x in lens for i in range(c["T"]))
    return {"bytes": unique * row + n * c["hq"] * (4 * dim + 4), "flops": 4.0 * pairs * c["hq"] * dim}


# ----------------------------------------------------------------- exact

def exact(case, seed):
    """The same results from the definitions, in 64 bits."""
    s, c = prepare(case, seed), case
    if c["op"] == "sample":
        return _exact_sample(s, c)
    lens, page = _lens(c), c["page"]
    hkv, dim = c["hkv"], c["dim"]
    table = s["block_table"].tolist()

    def rows(n, r, stop):
        """Rows [0, stop) of request r's k or v: [stop, heads, dim]."""
        at = torch.tensor(table[r][:-(-stop // page)], device="cuda")
        x = s[n].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() if c["e4m3"] else s[n][at].double()
        if c["e4m3"]:
            x = x * s[n + "_scale"][at].double()[..., None]
        return x.permute(0, 2, 1, 3).reshape(-1, hkv, dim)[:stop]

    if c["op"] == "read":
        return {n: torch.cat([rows(n, r, lens[r]) for r in range(c["R"])]) for n in ("k", "v")}

    if c["op"] == "attend":
        T, G = c["T"], c["hq"] // hkv
        out, lse = [], []
        for r in range(c["R"]):
            q = s["q"][r * T:(r + 1) * T].double().view(T, hkv, G, dim)
            k, v = rows("k", r, lens[r]), rows("v", r, lens[r])
            for i in range(T):
                n = lens[r] - T + i + 1
                a = torch.einsum("hgd,lhd->hgl", q[i], k[:n]) / math.sqrt(dim)
                z = torch.logsumexp(a, -1)
                lse.append(z.reshape(-1))
                out.append(torch.einsum("hgl,lhd->hgd", torch.exp(a - z[..., None]), v[:n]).reshape(c["hq"], dim))
        return {"out": torch.stack(out), "lse": torch.stack(lse)}

    # append: the angle of channel pair j at position p is p * 10000^(-2j / rot)
    T, rot, hq = c["T"], c["rot"], c["hq"]
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    first = 2 * j.long() if c["interleaved"] else j.long()
    second = first + 1 if c["interleaved"] else first + rot // 2
    result = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale") if n in s}
    qs = []
    for r in range(c["R"]):
        x = s["qkv"][r * T:(r + 1) * T].double()
        p = torch.arange(lens[r] - T, lens[r], device="cuda")
        a = (p.double()[:, None] * torch.exp(-math.log(10000.0) * 2.0 * j / rot))[:, None]
        y = x.clone()
        n = hq + hkv
        y[:, :n, first] = x[:, :n, first] * a.cos() - x[:, :n, second] * a.sin()
        y[:, :n, second] = x[:, :n, second] * a.cos() + x[:, :n, first] * a.sin()
        qs.append(y[:, :hq])
        at = torch.tensor(table[r], device="cuda")[p // page]
        for n, new in (("k", y[:, hq:hq + hkv]), ("v", y[:, hq + hkv:])):
            if c["e4m3"]:  # the values before their rounding to e4m3
                scale = new.abs().amax(-1) / E4M3_MAX
                result[n][at, :, p % page] = new / scale[..., None]
                result[n + "_scale"][at, :, p % page] = scale
            else:
                result[n][at, :, p % page] = new
    return {"q": torch.cat(qs), **result}


def _exact_sample(s, c):
    """The probability of each drawn token among those kept (tokens themselves are whole numbers)."""
    prob = []
    for row, u in zip(s["logits"].double().cpu(), s["u"].tolist()):
        if c["temperature"] <= 0:
            prob.append(1.0)
            continue
        p = torch.softmax(row / c["temperature"], 0)
        v, order = torch.sort(p, descending=True, stable=True)
        if c["top_k"]:
            v, order = v[:c["top_k"]], order[:c["top_k"]]
        if c["top_p"] < 1.0:
            n = max(1, int((torch.cumsum(v, 0) - v < c["top_p"] * v.sum()).sum()))
            v, order = v[:n], order[:n]
        if c["min_p"] > 0.0:
            v = v * (v >= c["min_p"] * p.max())
        kept = torch.zeros_like(p).scatter_(0, order, v)
        cum = kept.cumsum(0)
        at = int((cum > u * cum[-1]).int().argmax())
        prob.append(float(kept[at] / cum[-1]))
    out = {"tokens": None, "prob": torch.tensor(prob, dtype=torch.float64)}
    return {**out, "accept": None, "next": None} if c["T"] > 1 else out
