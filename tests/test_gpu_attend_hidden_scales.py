"""Value scales of keys that a query row does not see."""
import pytest

from test_gpu_attend import Problem

pytestmark = pytest.mark.gpu

CASES = [  # R, T, hq, hkv, dim, page, lens, prefix
    (1, 2, 6, 2, 128, 16, [70], 0),                      # 6 query rows
    (2, 8, 4, 2, 64, 32, [130, 1000], 0),                # 16 rows; the block across a tile's end
    (2, 16, 12, 2, 128, 64, [300, 136], 0),              # 96 rows
    (1, 16, 6, 1, 64, 64, [77], 0),
    (1, 50, 6, 1, 128, 32, [400], 0),                    # 300 rows
    (3, 5, 12, 2, 128, 32, [700, 520, 1000], 512),       # behind a prefix
]


@pytest.mark.parametrize("scale", [1e2, 1e8, 1e30])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_later_tokens_value_scale_does_not_reach_earlier_ones(dev, w12mod, case, scale):
    """The newest token's values are large and finite; the tokens before it give
    the bits that they give without."""
    import torch
    c = CASES[case]
    p = Problem(w12mod, dev, *c[:6], True, c[6], c[7])
    clean, z = p.run()
    p.check(clean, z, floor=2.0 ** -22)
    for r, n in enumerate(p.lens):
        p.kv.v_scale[int(p.table[r, (n - 1) // p.page]), :, (n - 1) % p.page] = scale
    out, lse = p.run()
    assert w12mod.get_device_error(p.ws) == 0
    shape = lambda t: t.reshape(p.R, p.T, -1)[:, :-1]  # noqa: E731
    assert torch.equal(shape(out.contiguous()), shape(clean.contiguous()))
    assert torch.equal(shape(lse), shape(z))
    assert scale < 1e30 or not torch.equal(out, clean)  # (the newest token's own weight may be tiny)
