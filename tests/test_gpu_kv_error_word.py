"""The error word of the cache calls is one int32."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["int8", "int64", "float32", "empty"])
def test_other_types_are_refused(dev, w12mod, kind):
    import torch
    kv = w12mod.KVCache.alloc(2, 1, 64, 16, w12mod.KV_BF16, dev)
    x = torch.zeros((1, 3, 64), dtype=torch.bfloat16, device=dev)
    q = torch.empty((1, 1, 64), dtype=torch.bfloat16, device=dev)
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    one = torch.ones(1, dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=dev)
    err = torch.zeros(0, dtype=torch.int32, device=dev) if kind == "empty" else torch.zeros(4, dtype=getattr(torch, kind), device=dev)
    with pytest.raises(ValueError):
        w12mod.kv_append(kv, x[:, :1], x[:, 1:2], x[:, 2:], table, one, 1, q, err_dev=err)
    with pytest.raises(ValueError):
        w12mod.kv_read(kv, table, cu, q, q.clone(), err_dev=err)
    for n in (1, 3):  # the first element is taken
        err = torch.zeros(n, dtype=torch.int32, device=dev)
        w12mod.kv_append(kv, x[:, :1], x[:, 1:2], x[:, 2:], table, one, 1, q, err_dev=err)
        w12mod.kv_read(kv, table, cu, q, q.clone(), err_dev=err)
        assert int(err.sum()) == 0
