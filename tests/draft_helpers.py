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
