"""Speculative decoding with a drafter of 4-bit weights and sampled verification.

The target is the decoder block of decode_step.py with its lossless W12 weights;
the drafter is the same block with the same matrices in 4 bits
(w12_fp4_encode), which draws T - 1 tokens per request and step, one at a time.
The target then sees the block of T tokens at once, and the drafts are accepted
against its probabilities (w12_verify_sampled), so that the text is distributed
as the target's own samples whatever the drafter is:

    T times: norm to e4m3 (w12_add_norm) -> 4-bit products on 8-bit tokens
    (w12_fp4_gemm_batched) -> rotary positions, cache, attention -> sample
    once:    the target's pass over T tokens -> w12_verify_sampled

as one CUDA graph a step.  (The drafter's T-th pass only brings its cache up to
the last draft; a refused token's cache rows are written over.)

    python examples/draft_step.py [--requests 8] [--prompt 1000] [--block 4] [--steps 32]
"""
import argparse
import os
import sys
import time

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [HERE, os.path.join(HERE, "..")]
from decode_step import DIM, HEADS, HIDDEN, KV_HEADS, PAGE, VOCAB, Block  # noqa: E402
from lossless_bit_weight_w12_gb300 import w12  # noqa: E402


class Drafter(Block):
    """A block's matrices in 4 bits; its normalised tokens in 8."""

    def __init__(self, target):
        self.dev, self.emb, self.rope = target.dev, target.emb, target.rope
        self.w = {}
        for name, bits in target.bits.items():
            w = torch.from_numpy(bits.view(np.int16)).to(self.dev).view(torch.bfloat16)
            self.w[name] = w12.FP4Weight.encode(w)

    def buffers(self, R, T, max_len, kv, prefix):
        b = super().buffers(R, T, max_len, kv, prefix)
        b["h"] = torch.empty(R * T, HIDDEN, dtype=torch.float8_e4m3fn, device=self.dev)
        b["h_scale"] = torch.empty(R * T, device=self.dev)
        return b

    def products_workspace(self, names, n):
        return w12.fp4_gemm_workspace_size([self.w[m] for m in names], n)

    def products(self, names, x, ys, ws):
        x, scale = x if isinstance(x, tuple) else (x, None)  # (attention's output is bf16)
        w12.FP4Batch([self.w[m] for m in names], [x] * len(names), ys, ws, None if scale is None else [scale] * len(names))()

    def norm(self, b, x, delta=None):
        w12.add_norm(x, None, b["h"], delta=delta, scale_out=b["h_scale"])
        return b["h"], b["h_scale"]


class Speculator:
    """R requests, each with a prompt of its own; step() commits 1 .. T tokens of each."""

    def __init__(self, target, drafter, prompts, T, max_new, temperature=0.8, top_p=0.95, seed=1):
        self.target, self.drafter, self.T = target, drafter, T
        R, P = prompts.shape
        dev = target.dev
        self.R, self.max_len = R, P + max_new + T
        blocks = -(-self.max_len // PAGE)
        self.table = torch.arange(R * blocks, dtype=torch.int32, device=dev).view(R, blocks)
        self.kv = [w12.KVCache.alloc(R * blocks, KV_HEADS, DIM, PAGE, device=dev) for _ in range(2)]
        for model, kv in zip((target, drafter), self.kv):  # the prompts, but for their last tokens
            for r in range(R):
                for at in range(0, P - 1, 128):
                    ids = torch.as_tensor(prompts[r, at:min(at + 128, P - 1)], device=dev)
                    n = len(ids)
                    b = model.buffers(1, n, at + n, kv, 0)
                    model.forward(b, kv, ids, self.table[r:r + 1], torch.tensor([at + n], dtype=torch.int32, device=dev), n,
                                  at + n, 0, logits=False)
        self.bt = target.buffers(R, T, self.max_len, self.kv[0], 0)
        self.bd = drafter.buffers(R, 1, self.max_len, self.kv[1], 0)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
        self.ids = torch.zeros(R, T, dtype=torch.int64, device=dev)  # the last committed token, then the drafts
        self.ids[:, 0] = torch.as_tensor(prompts[:, -1], device=dev)
        self.kv_len = torch.full((R,), P - 1 + T, dtype=torch.int32, device=dev)
        self.len1 = i32(R)
        self.draft, self.token, self.accept, self.next = i32(R, T - 1), i32(R), i32(R), i32(R)
        self.draft_logits = torch.empty(R, T - 1, VOCAB, device=dev)
        self.ratio = torch.empty(R, T - 1, device=dev)
        self.u = torch.empty(2, R, T, device=dev)  # for the drafts, for the verification
        full = lambda v: torch.full((R,), v, device=dev)  # noqa: E731
        self.temperature, self.top_p = full(temperature), full(top_p)
        self.cut = w12.Cut(temperature=self.temperature, top_p=self.top_p)
        self.ws = [w12.workspace(w12.sample_workspace_size(R, 1, VOCAB), dev),
                   w12.workspace(w12.verify_sampled_workspace_size(R, T, VOCAB), dev)]
        self.rng = torch.Generator(device=dev)
        self.rng.manual_seed(seed)
        self.graph = None

    def _pass(self):
        R, T = self.R, self.T
        for i in range(T):
            self.len1.copy_(self.kv_len - (T - 1 - i))
            self.drafter.forward(self.bd, self.kv[1], self.ids[:, i], self.table, self.len1, 1, self.max_len, 0,
                                 logits=i < T - 1)
            if i == T - 1:
                break
            w12.sample(self.bd["logits"], R, 1, self.u[0, :, i].contiguous(), self.token, self.ws[0], self.temperature,
                       top_p=self.top_p)
            self.draft_logits[:, i] = self.bd["logits"]
            self.draft[:, i] = self.token
            self.ids[:, i + 1] = self.token
        self.target.forward(self.bt, self.kv[0], self.ids.view(-1), self.table, self.kv_len, T, self.max_len, 0)
        w12.verify_sampled(self.bt["logits"], self.draft_logits.view(R * (T - 1), VOCAB), R, T, self.draft, self.u[1], self.accept,
                           self.next, self.ws[1], self.cut, self.cut, self.ratio)

    def step(self, graph=True):
        """(accepted drafts [R], next token [R], drafts [R, T - 1])."""
        self.u.uniform_(generator=self.rng)
        if graph and self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self._pass()  # (loads what a first call loads; writes what the graph writes)
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._pass()
        self.graph.replay() if graph else self._pass()
        out = [t.cpu().numpy() for t in (self.accept, self.next, self.draft)]
        self.ids[:, 0] = self.next.long()
        self.kv_len += self.accept + 1  # the block starts again behind the last accepted token
        return out

    def check(self):
        for ws in (*self.bt["ws"], *self.bd["ws"], *self.ws):
            assert w12.get_device_error(ws) == w12.OK


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--prompt", type=int, default=1000)
    p.add_argument("--block", type=int, default=4, help="tokens per request and step (1 committed, the others drafted)")
    p.add_argument("--steps", type=int, default=32)
    a = p.parse_args(argv)
    target = Block(torch.device("cuda:0"))
    prompts = np.random.default_rng(0).integers(0, VOCAB, (a.requests, a.prompt))
    s = Speculator(target, Drafter(target), prompts, a.block, a.steps * a.block)
    committed, t0 = 0, None
    for i in range(a.steps):
        acc, _, _ = s.step()
        if i == 0:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        committed += int(acc.sum()) + a.requests
    s.check()
    ms = (time.perf_counter() - t0) / max(a.steps - 1, 1) * 1e3
    print(f"{a.requests} requests, blocks of {a.block}: {committed} tokens in {a.steps} steps, "
          f"{committed / a.steps / a.requests:.2f} per request and step, {ms:.3f} ms a step with the host's part")
    return committed


if __name__ == "__main__":
    main()
