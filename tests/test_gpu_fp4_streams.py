"""FP4Weight on a stream that is not the current one: its buffers are that
stream's, so what is still to run on the current stream does not touch them."""
import numpy as np
import pytest

import draft_helpers as dh

pytestmark = pytest.mark.gpu


def _busy(torch, dev):
    big = torch.randn(6144, 6144, device=dev)
    for _ in range(10):
        big = (big @ big).clamp(-1, 1)
    return big


@pytest.mark.parametrize("call", ["encode", "pack", "decode"])
def test_buffers_belong_to_the_stream(dev, w12mod, call):
    import torch
    rng = np.random.default_rng(5)
    K, N = 1024, 2048
    codes, scales = dh.fp4_random(rng, K, N)
    codes_d, scales_d = torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev).view(torch.float8_e4m3fn)
    w = torch.from_numpy((0.02 * rng.standard_normal((N, K))).astype(np.float32)).to(dev, torch.bfloat16)
    packed, encoded = w12mod.FP4Weight.pack(codes_d, scales_d, 0.01), w12mod.FP4Weight.encode(w, 0.01)
    want = (encoded if call == "encode" else packed).decode()
    size = 4 * N * K if call == "decode" else int(w12mod.lib().w12_fp4_bytes(K, N)) + 256
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = _busy(torch, dev)
    late = torch.empty(size, dtype=torch.uint8, device=dev)
    late.fill_(0x3F)  # (runs after the products; its memory is the allocator's again at once)
    del late
    if call == "encode":
        got = w12mod.FP4Weight.encode(w, 0.01, stream=side)
    elif call == "pack":
        got = w12mod.FP4Weight.pack(codes_d, scales_d, 0.01, stream=side)
    else:
        got = packed.decode(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got if call == "decode" else got.decode(), want)
    del keep
