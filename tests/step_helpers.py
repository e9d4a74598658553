"""Plain 64-bit forms of the paged cache's rules, for the decode-step tests."""
import numpy as np

E4M3_MAX = 448.0


def rope_freqs(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def rotate(x, pos, rot, interleaved, base=10000.0):
    """x [tokens, heads, dim] float64 turned at positions pos [tokens]."""
    y = x.copy()
    if rot == 0:
        return y
    a = (np.asarray(pos, dtype=np.float64)[:, None] * rope_freqs(rot, base))[:, None, :]
    i0 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    y[..., i0] = x[..., i0] * np.cos(a) - x[..., i1] * np.sin(a)
    y[..., i1] = x[..., i1] * np.cos(a) + x[..., i0] * np.sin(a)
    return y


def pages(rng, lens, page, shared=0, spare=2):
    """(block_table [R, blocks] int32, n_pages): random page ids; the first
    `shared` pages of every request are the same."""
    need = [-(-max(n, 0) // page) for n in lens]
    own = [max(n - shared, 0) for n in need]
    ids = rng.permutation(shared + sum(own) + spare).astype(np.int32)
    table = np.zeros((len(lens), max(max(need), shared, 1)), dtype=np.int32)
    at = shared
    for r, n in enumerate(need):
        table[r, :shared] = ids[:shared]
        table[r, shared:shared + own[r]] = ids[at:at + own[r]]
        at += own[r]
    return table, len(ids)


def cache_values(kv):
    """k and v of a KVCache as float64 [n_pages, heads, page, dim] (host)."""
    out = []
    for t, s in ((kv.k, kv.k_scale), (kv.v, kv.v_scale)):
        x = t.float().cpu().numpy().astype(np.float64)
        out.append(x if s is None else x * s.cpu().numpy().astype(np.float64)[..., None])
    return out


def request_rows(values, table, r, n, page):
    """Rows 0 .. n - 1 of request r: [n, heads, dim]."""
    at = np.asarray(table[r][:-(-n // page)], dtype=np.int64)
    x = values[at].transpose(0, 2, 1, 3)
    return x.reshape(-1, *x.shape[2:])[:n]
