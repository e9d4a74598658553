"""Attention over the paged cache against its definition in 64 bits.

Tolerances.  Let u = 2^-8 (rounding to bf16), s the largest |score| of a row
and A = sum_j p_j |v_j| (p the softmax): a score is a sum of head_dim exact
products in fp32 (error at most head_dim 2^-24 scale |q|.|k|, below 2^-17
(1 + sum |q k| scale) for the sizes here), so a weight is off by a factor
1 + 2^-16 (1 + sum |q k| scale) and the weight entering the second product is
rounded by u at most (bf16 cache) or 2^-11 (e4m3 cache, fp16).  The output is
then within (u + 2^-10) A of the definition before its own rounding, u |out|
with it.  lse carries the scores' errors and fp32 roundings of its own size.
"""
import numpy as np
import pytest

from step_helpers import cache_values, pages, request_rows

pytestmark = pytest.mark.gpu


def _dev(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


class Problem:
    def __init__(self, w12, dev, R, T, hq, hkv, dim, page, e4m3, lens, prefix=0, seed=0, qscale=2.0):
        import torch
        rng = np.random.default_rng(seed + R * 100 + T * 10 + dim + page + len(lens))
        self.w12, self.dev, self.R, self.T, self.hq, self.hkv, self.dim, self.page = w12, dev, R, T, hq, hkv, dim, page
        self.lens, self.prefix = list(lens), prefix
        # the pages of the prefix (its last one, part of it, too) as every request's own table has them
        self.table, self.n_pages = pages(rng, [max(n, prefix) for n in lens], page, prefix // page)
        kv = self.kv = w12.KVCache.alloc(self.n_pages, hkv, dim, page, w12.KV_E4M3 if e4m3 else w12.KV_BF16, dev)
        for t in (kv.k, kv.v):
            t.copy_(_dev(rng.standard_normal(t.shape).astype(np.float32) * (60.0 if e4m3 else 1.0), dev).to(t.dtype))
        for t in (kv.k_scale, kv.v_scale):
            if t is not None:
                t.copy_(_dev((np.exp(rng.standard_normal(t.shape)) / 60.0).astype(np.float32), dev))
        if prefix % page:  # every request's copy of the page that the prefix ends in
            at, stop = self.table[:, prefix // page], prefix % page
            for t in (kv.k, kv.v, kv.k_scale, kv.v_scale):
                if t is not None:
                    for p in at[1:]:
                        t.view(torch.uint8 if e4m3 and t.dim() == 4 else t.dtype)[int(p), :, :stop] = \
                            t.view(torch.uint8 if e4m3 and t.dim() == 4 else t.dtype)[int(at[0]), :, :stop]
        q = rng.standard_normal((R * T, hq + 1, dim)).astype(np.float32) * qscale  # a wider token stride
        self.q_all = _dev(q, dev).to(torch.bfloat16)
        self.q = self.q_all[:, :hq]

    def poison(self):
        """NaN in every row that no request has: page tails, spare pages."""
        import torch
        kv = self.kv
        used = np.zeros((self.n_pages, self.page), dtype=bool)
        for r, n in enumerate(self.lens):
            for p in range(0, n):
                used[self.table[r, p // self.page], p % self.page] = True
        dead = _dev(~used, self.dev)[:, None, :].expand(-1, self.hkv, -1)
        for t in (kv.k, kv.v):
            if t.dtype == torch.bfloat16:
                t[dead] = float("nan")
            else:
                t.view(torch.uint8)[dead] = 0x7F
        for t in (kv.k_scale, kv.v_scale):
            if t is not None:
                t[dead] = float("nan")

    def run(self, ws=None, lse=True, max_len=None, table=None, stream=None):
        import torch
        n = self.R * self.T
        out_all = torch.full((n, self.hq + 2, self.dim), 5.0, dtype=torch.bfloat16, device=self.dev)
        out = out_all[:, 1:1 + self.hq]
        z = torch.full((n, self.hq), 5.0, device=self.dev) if lse else None
        m = max(self.lens + [0]) if max_len is None else max_len
        self.ws = self.w12.workspace(self.w12.attend_workspace_size(self.kv, self.R, self.T, self.hq, m, self.prefix),
                                     self.dev) if ws is None else ws
        self.w12.attend(self.kv, self.q, _dev(self.table, self.dev) if table is None else table,
                        _dev(np.array(self.lens, np.int32), self.dev), self.T, m, out, self.ws,
                        prefix_len=self.prefix, lse_dev=z, stream=stream)
        assert bool((out_all[:, 0] == 5.0).all()) and bool((out_all[:, -1] == 5.0).all())
        return out, z

    def check(self, out, lse, rows=None, floor=0.0):
        q = self.q.float().cpu().numpy().astype(np.float64)
        out = out.float().cpu().numpy().astype(np.float64)
        lse = None if lse is None else lse.cpu().numpy().astype(np.float64)
        kvals, vvals = cache_values(self.kv)
        G, scale, u = self.hq // self.hkv, self.dim ** -0.5, 2.0 ** -8
        e4m3 = self.kv.k_scale is not None
        for r in range(self.R):
            n = self.lens[r]
            k, v = request_rows(kvals, self.table, r, n, self.page), request_rows(vvals, self.table, r, n, self.page)
            for i in range(self.T):
                tok, stop = r * self.T + i, max(n - self.T + i + 1, 0)
                if rows is not None and tok not in rows:
                    continue
                for h in range(self.hkv):
                    at = slice(h * G, (h + 1) * G)
                    if stop == 0:
                        assert np.all(out[tok, at] == 0.0)
                        assert lse is None or np.all(np.isneginf(lse[tok, at]))
                        continue
                    s = q[tok, at] @ k[:stop, h].T * scale
                    size = (np.abs(q[tok, at]) @ np.abs(k[:stop, h]).T * scale).max(-1)
                    m = s.max(-1, keepdims=True)
                    p = np.exp(s - m)
                    l = p.sum(-1, keepdims=True)
                    want = p @ v[:stop, h] / l
                    amount = p @ np.abs(v[:stop, h]) / l
                    w = 2.0 ** -11 if e4m3 else u
                    tol = (w + 2.0 ** -16 * (1 + size[:, None])) * amount + u * np.abs(want) + 1e-30 + floor * stop * np.abs(v[:stop, h]).max()
                    err = np.abs(out[tok, at] - want)
                    assert np.all(err <= tol * (1 + u)), (tok, h, float((err / tol).max()))
                    if lse is not None:
                        z = (m + np.log(l))[:, 0]
                        assert np.all(np.abs(lse[tok, at] - z) <= 2.0 ** -17 * (1 + size) + 2.0 ** -22 * np.abs(z))


CASES = [  # R, T, hq, hkv, dim, page, lens, prefix
    (1, 1, 1, 1, 128, 16, [1], 0),
    (1, 1, 6, 1, 128, 64, [63], 0),
    (1, 1, 6, 1, 64, 64, [64], 0),
    (1, 1, 8, 8, 64, 32, [65], 0),
    (4, 1, 48, 8, 128, 64, [1, 300, 2500, 777], 0),
    (3, 1, 15, 1, 128, 128, [500, 129, 128], 0),
    (2, 3, 6, 2, 128, 16, [3, 200], 0),
    (2, 16, 12, 2, 128, 64, [16, 517], 0),          # 96 query rows a head
    (2, 16, 12, 2, 64, 32, [40, 1000], 0),
    (3, 5, 7, 1, 64, 128, [2, 5, 130], 0),          # 35 rows; a request with fewer than T tokens
    (5, 4, 4, 2, 128, 16, [0, 1, 3, 4, 90], 0),     # rows without keys
    (1, 130, 2, 1, 128, 32, [200], 0),              # a piece of a prompt
    (4, 1, 6, 1, 128, 64, [700, 640, 641, 900], 640),   # the prefix alone, and one key more
    (7, 1, 12, 2, 128, 32, [333, 400, 334, 1000, 350, 360, 500], 333),  # ends inside a page and a tile
    (6, 4, 12, 2, 64, 16, [210, 204, 300, 220, 250, 1204], 200),
    (9, 16, 6, 1, 128, 64, [1100 + 50 * i for i in range(9)], 1050),    # 864 rows under the prefix
    (3, 2, 4, 1, 128, 128, [100, 64, 300], 90),     # a request that ends inside the prefix
    (70, 1, 8, 2, 64, 16, [130 + 3 * i for i in range(70)], 129),
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) + "-" + str(c[:6]).replace(" ", "") for i, c in enumerate(CASES)])
def test_attend(dev, w12mod, case, e4m3):
    import torch
    p = Problem(w12mod, dev, *case[:6], e4m3, case[6], case[7])
    p.poison()
    out, lse = p.run()
    assert w12mod.get_device_error(p.ws) == 0
    p.check(out, lse)
    again, z = p.run(ws=p.ws)  # a used workspace: the same bits
    assert torch.equal(out, again) and torch.equal(lse, z)
    third, _ = p.run(lse=False, max_len=max(p.lens) + 1000)
    assert third is not None and bool((third.float() - out.float()).abs().max() <= 2.0 ** -6 * out.float().abs().max() + 1e-30)


BLOCKS = [
    (3, 50, 6, 1, 64, 16, [0, 49, 640], 0),         # 300 rows: none, some and all with keys
    (4, 12, 6, 2, 128, 64, [128, 139, 140, 1035], 0),  # the new tokens before, across and after a tile's end
    (5, 7, 12, 2, 128, 32, [700, 520, 519, 640, 1000], 512),  # 42 rows after a prefix
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", BLOCKS, ids=[str(i) for i in range(len(BLOCKS))])
def test_blocks_at_tile_ends(dev, w12mod, case, e4m3):
    """fp16 weights have a floor: spacing 2^-24, where the largest weight times
    its scale is 2^7 (2^e the bound of a tile's scales, m = max - 7 + e).  A
    weight is thus off by up to 2^-25 2^(e - 7) <= 2^-31 max(scale) of the
    row's largest, and an output by 2^-31 max(scale) max(code) per key, whose
    product is at most 2^9 max |v| here (scales and codes apart by no more)."""
    p = Problem(w12mod, dev, *case[:6], e4m3, case[6], case[7])
    p.poison()
    out, lse = p.run()
    assert w12mod.get_device_error(p.ws) == 0
    p.check(out, lse, floor=2.0 ** -22 if e4m3 else 0.0)


def test_prefix_and_plain_agree(dev, w12mod):
    """The same requests with the prefix taken apart and as part of each request."""
    p = Problem(w12mod, dev, 5, 2, 12, 2, 128, 32, False, [500, 520, 600, 700, 801], 480)
    a, _ = p.run()
    p.check(a, None)
    p.prefix = 0
    b, _ = p.run()
    p.check(b, None)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_later_tokens_do_not_leak(dev, w12mod, e4m3):
    """NaN and infinities in the key and value of the draft block's later
    tokens reach no earlier token; the tokens that see them get them."""
    import torch
    T, n = 8, 100
    p = Problem(w12mod, dev, 1, T, 6, 1, 128, 16, e4m3, [n])
    clean, _ = p.run()
    at = n - 3  # position of token T - 3
    pg, row = int(p.table[0, at // 16]), at % 16
    for what in ("v", "k"):
        t = getattr(p.kv, what)
        keep = t.clone()
        if e4m3:
            t.view(torch.uint8)[pg, 0, row, 7] = 0x7F
        else:
            t[pg, 0, row, 7] = float("inf") if what == "v" else float("nan")
        out, _ = p.run()
        assert torch.equal(out[:T - 3], clean[:T - 3])
        bad = out[T - 3:].float()
        if what == "v":
            assert not bool(torch.isfinite(bad[:, :, 7]).any())
            fine = torch.cat([bad[:, :, :7], bad[:, :, 8:]], -1)
            ref = clean[T - 3:].float()
            # the other channels of the odd row were kept out of the matrix product too: within its tolerance
            assert bool(((fine - torch.cat([ref[:, :, :7], ref[:, :, 8:]], -1)).abs() <= 2.0 ** -6).all())
        else:
            assert bool(torch.isnan(bad).all())
        t.copy_(keep)
    if e4m3:
        for s in (p.kv.k_scale, p.kv.v_scale):
            keep = s.clone()
            s[pg, 0, row] = float("nan")
            out, _ = p.run()
            assert torch.equal(out[:T - 3], clean[:T - 3]) and bool(torch.isnan(out[T - 3:]).all())
            s.copy_(keep)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,hq,n", [(2, 6, 90), (2, 6, 1000), (4, 6, 90), (4, 6, 1000), (40, 6, 300), (40, 6, 128), (130, 1, 131)])
def test_odd_values_of_any_block(dev, w12mod, T, hq, n, e4m3):
    """As above for few rows, several tiles, more than 128 rows; values that are
    not finite in several channels, in the first new token and in the last."""
    import torch
    p = Problem(w12mod, dev, 1, T, hq, 1, 128, 32, e4m3, [n])
    clean, _ = p.run()
    spots = [(n - T + 1, 3), (n - T + 1, 4), (n - T // 2, 127), (n - 1, 64)]  # position, channel
    t = p.kv.v
    for at, ch in spots:
        if e4m3:
            t.view(torch.uint8)[int(p.table[0, at // 32]), 0, at % 32, ch] = 0x7F
        else:
            t[int(p.table[0, at // 32]), 0, at % 32, ch] = float("-inf")
    out, lse = p.run()
    again, _ = p.run()
    assert torch.equal(torch.isfinite(out), torch.isfinite(again))
    hit = torch.zeros(T, 128, dtype=torch.bool)
    for at, ch in spots:
        hit[at - (n - T):, ch] = True
    hit = hit[:, None, :].expand(-1, hq, -1)
    got = out.float().cpu()
    assert not bool(torch.isfinite(got[hit]).any()) and bool(torch.isfinite(got[~hit]).all())
    assert bool(((got - clean.float().cpu())[~hit].abs() <= 2.0 ** -6).all())
    assert bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_lowest_scores_and_large_ones(dev, w12mod, e4m3):
    """Scores at -inf, all equal, and far apart (one key takes everything)."""
    import torch
    p = Problem(w12mod, dev, 1, 1, 2, 1, 64, 16, e4m3, [300], qscale=300.0)
    out, lse = p.run()
    p.check(out, lse)
    p.q_all.zero_()  # all scores equal: the mean of the values
    out, lse = p.run()
    p.check(out, lse)
    if not e4m3:
        p.q_all.fill_(1.0)
        p.kv.k.fill_(float("-inf"))  # every score is -inf: no key counts
        out, lse = p.run()
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_long_context_offsets(dev, w12mod):
    """Pages at the end of a cache whose element offsets pass 2^32, and 40000 keys."""
    import torch
    page, hkv, dim, n = 128, 8, 128, 40000
    n_pages = (1 << 32) // (dim * page * hkv) + 400
    kv = w12mod.KVCache.alloc(n_pages, hkv, dim, page, w12mod.KV_E4M3, dev)
    blocks = -(-n // page)
    table = torch.arange(n_pages - 1, n_pages - 1 - blocks, -1, dtype=torch.int32, device=dev)[None]
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    ids = table[0].long()
    for t, s in ((kv.k, kv.k_scale), (kv.v, kv.v_scale)):
        x = 50 * torch.randn(blocks, hkv, page, dim, generator=g, device=dev)
        t.view(torch.uint8)[ids] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        s[ids] = 0.02
    q = torch.randn(1, 48, dim, generator=g, device=dev).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(1, 48, device=dev)
    ws = w12mod.workspace(w12mod.attend_workspace_size(kv, 1, 1, 48, n), dev)
    w12mod.attend(kv, q, table, torch.tensor([n], dtype=torch.int32, device=dev), 1, n, out, ws, lse_dev=lse)
    k, v = (t.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * 0.02 for t in (kv.k, kv.v))
    k, v = (x.transpose(0, 1).reshape(hkv, -1, dim)[:, :n] for x in (k, v))
    sc = torch.einsum("hgd,hnd->hgn", q.double().view(hkv, 6, dim), k) * dim ** -0.5
    pr = torch.softmax(sc, -1)
    want = torch.einsum("hgn,hnd->hgd", pr, v).reshape(48, dim)
    amount = torch.einsum("hgn,hnd->hgd", pr, v.abs()).reshape(48, dim)
    assert bool(((out[0].double() - want).abs() <= 2.0 ** -10 * amount + 2.0 ** -8 * want.abs()).all())
    assert bool(((lse[0].double() - torch.logsumexp(sc, -1).reshape(-1)).abs() <= 2.0 ** -15).all())


def test_one_workspace_for_all_sizes(dev, w12mod):
    """A workspace used for one size serves any other that fits, back and forth."""
    shapes = [(4, 1, 48, 8, 128, 64, [1, 300, 2500, 777], 0), (2, 16, 12, 2, 128, 64, [16, 517], 0),
              (1, 130, 2, 1, 128, 32, [2000], 0), (7, 1, 12, 2, 128, 32, [333, 400, 334, 1000, 350, 360, 500], 333),
              (1, 1, 6, 1, 128, 64, [9000], 0)]
    probs = [Problem(w12mod, dev, *c[:6], e4m3, c[6], c[7]) for c in shapes for e4m3 in (False, True)]
    need = max(w12mod.attend_workspace_size(p.kv, p.R, p.T, p.hq, max(p.lens), p.prefix) for p in probs)
    ws = w12mod.workspace(need, dev)
    for p in probs + probs[::-1]:
        out, lse = p.run(ws=ws)
        p.check(out, lse)
    assert w12mod.get_device_error(ws) == 0


def test_device_errors(dev, w12mod):
    """Lengths above max_len or the table, and pages outside the cache: told in
    the workspace's error word, which get_device_error clears."""
    import torch
    p = Problem(w12mod, dev, 2, 1, 4, 2, 64, 16, False, [100, 200])
    out, _ = p.run(max_len=150)
    assert w12mod.get_device_error(p.ws) == w12mod.ERR_DEVICE
    p.check(out, None, rows=[0])
    table = _dev(p.table, dev)
    table[1, 3] = p.n_pages
    out, _ = p.run(table=table)
    assert w12mod.get_device_error(p.ws) == w12mod.ERR_DEVICE
    p.check(out, None, rows=[0])
    out, _ = p.run(table=_dev(p.table, dev)[:, :8].contiguous())  # 128 rows of table for 200 keys
    assert w12mod.get_device_error(p.ws) == w12mod.ERR_DEVICE
    p.check(out, None, rows=[0])
    out, lse = p.run()
    assert w12mod.get_device_error(p.ws) == 0
    p.check(out, lse)


def test_other_stream_and_graph(dev, w12mod):
    """On a side stream, and captured once and replayed with new lengths."""
    import torch
    p = Problem(w12mod, dev, 3, 1, 6, 1, 128, 64, False, [100, 500, 900])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, lse = p.run()
        s.synchronize()
        p.check(out, lse)
        table, lens = _dev(p.table, dev), _dev(np.array(p.lens, np.int32), dev)
        q = p.q.contiguous()
        g_out, g_lse = torch.empty_like(q), torch.empty(3, 6, device=dev)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            w12mod.attend(p.kv, q, table, lens, 1, 900, g_out, p.ws, lse_dev=g_lse)
        for new in ([100, 500, 900], [1, 64, 0], [100, 65, 899]):
            lens.copy_(_dev(np.array(new, np.int32), dev))
            graph.replay()
            s.synchronize()
            p.lens = new
            p.check(g_out, g_lse)
