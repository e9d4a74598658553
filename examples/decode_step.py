"""One decoder block served with W12 weights, a paged cache and sampled draft blocks.

Requests share a prompt.  The prompt goes once through the block in pieces and
into pages that every request's block table names; then each step runs a draft
block of T tokens per request:

    projections (w12_gemm_batched) -> rotary positions and cache (w12_kv_append)
    -> attention, the prompt read once for all requests (w12_attend)
    -> output projection, lm_head (w12_gemm) -> sampled tokens and how many of
    the draft they accept (w12_sample)

as one CUDA graph.  A rejected token's cache rows are simply written over: a
request's length goes back to its last accepted token.

    python examples/decode_step.py [--requests 8] [--prompt 1000] [--block 4] [--steps 32] [--e4m3]

Weights are random (seeded), so the text is noise; the drafts are the tokens
that followed the same token before.
"""
import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from lossless_bit_weight_w12_gb300 import synth, w12  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, VOCAB, PAGE = 1024, 12, 2, 128, 8192, 64
POSITIONS = 8192


def norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Block:
    """The weights (encoded once) and what a pass of n tokens needs."""

    def __init__(self, dev, seed=0):
        rng = synth.streams(seed, 6)
        self.dev = dev
        shapes = (("q", HIDDEN, HEADS * DIM), ("k", HIDDEN, KV_HEADS * DIM), ("v", HIDDEN, KV_HEADS * DIM),
                  ("o", HEADS * DIM, HIDDEN), ("lm_head", HIDDEN, VOCAB))
        self.bits, self.w = {}, {}
        for r, (name, k, n) in zip(rng, shapes):
            self.bits[name] = synth.weights(r, k, n)
            d, blob = w12.encode(self.bits[name], w12.LAYOUT_NK)
            self.w[name] = (d, w12.upload(blob, dev))
        emb = rng[5].standard_normal((VOCAB, HIDDEN)).astype(np.float32)
        self.emb = torch.from_numpy(emb).to(dev).to(torch.bfloat16)
        self.rope = torch.from_numpy(w12.rope_table(POSITIONS, DIM)).to(dev)

    def buffers(self, R, T, max_len, kv, prefix):
        """Outputs and workspaces of passes of R x T tokens."""
        n, dev, b = R * T, self.dev, {}
        f32 = lambda *s: torch.empty(*s, device=dev)  # noqa: E731
        b["q"], b["k"], b["v"] = f32(n, HEADS * DIM), f32(n, KV_HEADS * DIM), f32(n, KV_HEADS * DIM)
        b["q16"] = torch.empty(n, HEADS, DIM, dtype=torch.bfloat16, device=dev)
        b["a"] = torch.empty(n, HEADS, DIM, dtype=torch.bfloat16, device=dev)
        b["o"], b["logits"] = f32(n, HIDDEN), f32(n, VOCAB)
        qkv = [self.w[m] for m in "qkv"]
        b["ws"] = [w12.workspace(w12.gemm_batched_workspace_size([d for d, _ in qkv], n), dev),
                   w12.workspace(w12.attend_workspace_size(kv, R, T, HEADS, max_len, prefix), dev),
                   w12.workspace(max(w12.gemm_workspace_size(self.w[m][0], n) for m in ("o", "lm_head")), dev)]
        return b

    def forward(self, b, kv, ids, table, kv_len, T, max_len, prefix, logits=True):
        """ids [R * T] -> b["logits"]; the tokens enter the cache at kv_len - T .. kv_len - 1."""
        x = self.emb[ids]
        h = norm(x)
        w12.gemm_batched([self.w[m][0] for m in "qkv"], [self.w[m][1] for m in "qkv"], [h] * 3,
                         [b["q"], b["k"], b["v"]], b["ws"][0])
        n = len(ids)
        w12.kv_append(kv, b["q"].view(n, HEADS, DIM), b["k"].view(n, KV_HEADS, DIM), b["v"].view(n, KV_HEADS, DIM),
                      table, kv_len, T, b["q16"], self.rope)
        w12.attend(kv, b["q16"], table, kv_len, T, max_len, b["a"], b["ws"][1], prefix_len=prefix)
        if not logits:
            return
        w12.gemm(*self.w["o"], b["a"].view(n, HEADS * DIM), b["o"], b["ws"][2])
        w12.gemm(*self.w["lm_head"], norm(x.float() + b["o"]), b["logits"], b["ws"][2])


class Server:
    """R requests under one prompt; step() commits 1 .. T tokens of each."""

    def __init__(self, block, prompt, R, T, max_new, e4m3=False, temperature=0.8, top_k=0, top_p=0.95, seed=1):
        dev, self.block, self.R, self.T = block.dev, block, R, T
        P = self.prompt_len = len(prompt)
        self.max_len = P + max_new + T
        shared, own = (P - 1) // PAGE, -(-self.max_len // PAGE) - (P - 1) // PAGE
        self.kv = w12.KVCache.alloc(shared + R * own, KV_HEADS, DIM, PAGE, w12.KV_E4M3 if e4m3 else w12.KV_BF16, dev)
        table = np.empty((R, shared + own), dtype=np.int32)
        table[:, :shared] = np.arange(shared)
        table[:, shared:] = shared + np.arange(R * own).reshape(R, own)
        self.table = torch.from_numpy(table).to(dev)
        # the prompt, but for its last token, in pieces through request 0's
        # table; its last page is part of each request's own
        for at in range(0, P - 1, 128):
            ids = torch.as_tensor(prompt[at:min(at + 128, P - 1)], device=dev)
            n = len(ids)
            b = block.buffers(1, n, at + n, self.kv, 0)
            block.forward(b, self.kv, ids, self.table[:1].contiguous(),
                          torch.tensor([at + n], dtype=torch.int32, device=dev), n, at + n, 0, logits=False)
        for t in (self.kv.k, self.kv.v, self.kv.k_scale, self.kv.v_scale):
            if t is not None:
                raw = t.view(torch.uint8) if e4m3 and t.dim() == 4 else t
                raw[self.table[1:, shared].long()] = raw[self.table[0, shared].long()].clone()
        self.b = block.buffers(R, T, self.max_len, self.kv, P - 1)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
        self.ids = torch.zeros(R, T, dtype=torch.int64, device=dev)      # last committed token, then the draft
        self.ids[:, 0] = int(prompt[-1])
        self.kv_len = torch.full((R,), P - 1 + T, dtype=torch.int32, device=dev)
        self.draft, self.tokens, self.accept, self.next = i32(R, max(T - 1, 1)), i32(R, T), i32(R), i32(R)
        self.u, self.prob = torch.empty(R * T, device=dev), torch.empty(R * T, device=dev)
        full = lambda v, d: torch.full((R,), v, dtype=d, device=dev)  # noqa: E731
        self.temperature = full(temperature, torch.float32)
        self.top_k = full(top_k, torch.int32) if top_k else None
        self.top_p = full(top_p, torch.float32) if top_p < 1 else None
        self.ws = w12.workspace(w12.sample_workspace_size(R, T, VOCAB), dev)
        self.rng = torch.Generator(device=dev)
        self.rng.manual_seed(seed)
        self.graph = None

    def _pass(self):
        R, T = self.R, self.T
        self.block.forward(self.b, self.kv, self.ids.view(-1), self.table, self.kv_len, T, self.max_len,
                           self.prompt_len - 1)
        w12.sample(self.b["logits"], R, T, self.u, self.tokens, self.ws, self.temperature, self.top_k, self.top_p,
                   prob_dev=self.prob, draft_dev=self.draft if T > 1 else None, accept_dev=self.accept,
                   next_dev=self.next)

    def step(self, draft=None, graph=True):
        """draft [R, T - 1]: guesses.  Returns (accepted drafts [R], next token [R], sampled tokens [R, T])."""
        R, T = self.R, self.T
        if T > 1:
            self.draft.copy_(draft)
            self.ids[:, 1:] = self.draft
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
        acc, nxt = self.accept.cpu(), self.next.cpu()
        tokens = self.tokens.cpu()
        self.ids[:, 0] = self.next.long()
        self.kv_len += self.accept + 1  # the block starts again behind the last accepted token
        return acc.numpy(), nxt.numpy(), tokens.numpy().reshape(R, T)

    def check(self):
        for ws in (self.b["ws"][0], self.b["ws"][1], self.b["ws"][2], self.ws):
            assert w12.get_device_error(ws) == w12.OK


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--prompt", type=int, default=1000)
    p.add_argument("--block", type=int, default=4, help="tokens per request and step (1 committed, the others drafted)")
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--e4m3", action="store_true", help="cache in e4m3 with a scale per token and head")
    a = p.parse_args(argv)
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(0)
    block = Block(dev)
    R, T = a.requests, a.block
    server = Server(block, rng.integers(0, VOCAB, a.prompt), R, T, a.steps * T, a.e4m3, temperature=0.05)
    seen = [{} for _ in range(R)]
    last = server.ids[:, 0].cpu().numpy()
    committed, t0 = 0, None
    for s in range(a.steps):
        draft = np.zeros((R, max(T - 1, 1)), dtype=np.int32)
        for r in range(R):
            tok = int(last[r])
            for i in range(T - 1):
                tok = draft[r, i] = seen[r].get(tok, 0)
        acc, nxt, tokens = server.step(torch.from_numpy(draft))
        if s == 0:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        for r in range(R):
            for tok in list(draft[r, :acc[r]]) + [nxt[r]]:
                seen[r][int(last[r])] = int(tok)
                last[r] = tok
        committed += int(acc.sum()) + R
    server.check()
    ms = (time.perf_counter() - t0) / max(a.steps - 1, 1) * 1e3
    print(f"{R} requests under a prompt of {a.prompt}, blocks of {T}: {committed} tokens in {a.steps} steps, "
          f"{committed / a.steps / R:.2f} per request and step, {ms:.3f} ms a step with the host's part")
    return committed


if __name__ == "__main__":
    main()
