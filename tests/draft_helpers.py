"""Plain 64-bit forms of the draft-model calls' rules, for their tests."""
import numpy as np

E4M3_MAX = 448.0


def bits_f64(t):
    """A float tensor's values as float64 (host)."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def add_norm(x, delta, weight, offset, eps):
    """(h, y) of float64 arrays [n, dim]."""
    h = x if delta is None else x + delta
    w = offset + (1.0 if weight is None else weight)
    return h, h * w / np.sqrt((h * h).mean(-1, keepdims=True) + eps)


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """Every e4m3 byte's value (NaN for 0x7F and 0xFF)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m / 8 * 2.0 ** -6)
    v[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -v, v)


def fp4_values(codes, scales, scale):
    """float64 [N, K] of codes uint8 [N, K / 2] and scale bytes uint8 [N, K / 16]."""
    n, half = codes.shape
    c = np.stack([codes & 15, codes >> 4], -1).reshape(n, -1)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    return (v.reshape(n, -1, 16) * e4m3_values()[scales][..., None]).reshape(n, -1) * float(np.float32(scale))


def fp4_random(rng, K, N):
    """(codes, scale bytes) of a random matrix; the scales spread over e4m3's range, zeros among them."""
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = rng.integers(0x20, 0x58, (N, K // 16)).astype(np.uint8)
    odd = rng.random(scales.shape)
    scales[odd < 0.02] = 0
    scales[(odd >= 0.02) & (odd < 0.06)] = rng.integers(1, 8)
    scales[odd > 0.98] |= 0x80
    return codes, scales


def fp4_encode(w, scale):
    """(codes [N, K], scale bytes) of float32 weights by w12_fp4_encode's rule, in fp32."""
    f = np.float32
    table = e4m3_values()[:127].astype(f)
    g = np.abs(w.astype(f)).reshape(w.shape[0], -1, 16)
    amax = g.max(-1)
    want = np.minimum((amax / (f(6) * f(scale))).astype(f), f(448))
    # nearest, ties to the even byte
    hi = np.clip(np.searchsorted(table, want), 1, 126)
    lo = hi - 1
    dl, dh = want.astype(np.float64) - table[lo], table[hi].astype(np.float64) - want
    s = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    s = np.where((s == 0) & (amax > 0), 1, s)
    inv = np.where(s > 0, f(1) / np.where(s > 0, table[s] * f(scale), f(1)), f(0)).astype(f)
    a = (g * inv[..., None]).astype(f)
    code = ((a > 0.25).astype(int) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code.reshape(w.shape), s.astype(np.uint8)
