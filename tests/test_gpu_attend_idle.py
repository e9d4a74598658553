"""Requests without keys (idle slots of a fixed batch) beside requests that
share a prefix."""
import numpy as np
import pytest

from test_gpu_attend import Problem, _dev

pytestmark = pytest.mark.gpu

CASES = [  # R, T, hq, hkv, dim, page, lens, prefix
    (4, 1, 6, 1, 128, 64, [700, 0, 641, 900], 640),
    (4, 1, 6, 1, 128, 64, [0, 0, 700, 900], 640),        # the first request is idle, too
    (6, 4, 12, 2, 64, 16, [0, 304, 400, 0, 350, 1204], 300),
    (9, 16, 6, 1, 128, 64, [0] + [1100 + 50 * i for i in range(7)] + [0], 1050),
    (70, 1, 8, 2, 64, 16, [0 if i % 3 == 0 else 130 + 3 * i for i in range(70)], 129),
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_idle_requests_do_not_part_the_prefix(dev, w12mod, case, e4m3):
    """The prefix's whole tiles are still read once, through the first request
    that has keys: the others' tables name no page there, and nothing is
    recorded.  Idle requests' queries and tables hold anything."""
    c = CASES[case]
    p = Problem(w12mod, dev, *c[:6], e4m3, c[6], c[7])
    p.poison()
    first = next(r for r in range(p.R) if p.lens[r])
    shared = min([c[7]] + [n - p.T + 1 for n in p.lens if n]) // 128 * 128
    assert shared > 0
    table = p.table.copy()
    for r in range(p.R):
        if p.lens[r] == 0:
            table[r] = [-1, p.n_pages, 1 << 30, -(1 << 31)][r % 4]
            p.q_all[r * p.T:(r + 1) * p.T] = float("nan")
        elif r != first:
            table[r, :shared // p.page] = -1
    out, lse = p.run(table=_dev(table, dev))
    assert w12mod.get_device_error(p.ws) == 0
    p.check(out, lse, floor=2.0 ** -22 if e4m3 else 0.0)


@pytest.mark.parametrize("T", [1, 16])
def test_all_idle(dev, w12mod, T):
    import torch
    p = Problem(w12mod, dev, 5, T, 6, 1, 128, 64, False, [0] * 5, 640)
    out, lse = p.run(max_len=1000, table=_dev(np.full_like(p.table, -1), dev))
    assert w12mod.get_device_error(p.ws) == 0
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
