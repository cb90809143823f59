"""Serving a few requests through one attention layer with a paged key/value
cache: prompts admitted together, then decoding one token per request and step,
with one request joining while the others decode.

    python examples/serve_paged.py [--width 4096] [--heads 32] [--kv-heads 8] [--four-bit]

Weights are random, INT8 in groups of 64; the "tokens" are random activations.
Every step runs kv_plan (block tables and slots on the GPU from the lengths),
and attn_layer_paged: the quantised projections, rope_append and attn_prompt or
attn_paged.  Prints what each step did, and checks the decoded rows against one
attn_prompt over each request's whole sequence.  --four-bit holds the cache in 4
bits (groups of 64), a little over a quarter of the memory: the difference is
then what that costs.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import group_quantized_moe_gb300 as lib  # noqa: E402


class Server:
    """One layer, its cache and block tables, and the requests' lengths."""

    def __init__(self, width, heads, kv_heads, head_dim, blocks=512, block_size=16, columns=64,
                 requests=8, max_seq=1024, dtype=torch.bfloat16, seed=0,
                 four_bit=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = (heads + 2 * kv_heads) * head_dim
        w = torch.randn(rows, width, device="cuda", generator=g) * width ** -0.5
        wo = torch.randn(width, heads * head_dim, device="cuda", generator=g) * (heads * head_dim) ** -0.5
        self.wqkv = lib.qmm_quantize_groupwise(w, 8, 64)
        self.wo = lib.qmm_quantize_groupwise(wo, 8, 64)
        self.heads, self.kv_heads, self.block_size = heads, kv_heads, block_size
        self.cos, self.sin = lib.rope_table(max_seq, head_dim)
        self.dtype = dtype
        self.cache = (lib.paged_kv4(blocks, kv_heads, block_size, head_dim) if four_bit else
                      lib.paged_kv(blocks, kv_heads, block_size, head_dim, dtype))
        self.free = torch.arange(blocks, dtype=torch.int32, device="cuda")
        self.table = torch.full((requests, columns), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def step(self, x, new_lens, prompts=False):
        """new_lens: new tokens of every request (host integers, summing to
        the rows of x).  Returns the layer's output rows."""
        new = torch.tensor(new_lens, dtype=torch.int32, device="cuda")
        plan = lib.kv_plan(self.lens, new, self.table, self.free, self.block_size, x.shape[0])
        y = lib.attn_layer_paged(x, self.wqkv, self.wo, self.heads, self.cos, self.sin, self.cache,
                                 plan, self.table, prompts=prompts)
        self.free = self.free[int(plan.blocks_used):]  # the host keeps the free list
        self.lens = plan.kv_lens
        return y

    def whole(self, x):
        """The same layer over one request's whole sequence, without the cache."""
        qkv = lib.qmm_linear_batched(x, self.wqkv)
        n = x.shape[0]
        q, k, v = lib.rope_append(qkv, self.heads, torch.arange(n, dtype=torch.int32, device="cuda"),
                                  None, self.cos, self.sin, None, keep_kv=True, n_kv=self.kv_heads,
                                  y_dtype=self.dtype)
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        a = lib.attn_prompt(q, k, v, cu, y_dtype=x.dtype)
        return lib.qmm_linear_batched(a.view(n, -1), self.wo)


def main(argv=None) -> float:
    ap = argparse.ArgumentParser()
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--four-bit", action="store_true")
    ap.add_argument("--quiet", action="store_true")
    a = ap.parse_args(argv)
    say = (lambda *s: None) if a.quiet else print
    s = Server(a.width, a.heads, a.kv_heads, a.head_dim, requests=4, four_bit=a.four_bit)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = lambda n: torch.randn(n, a.width, device="cuda", generator=g).bfloat16()
    seen = [[] for _ in range(4)]  # every request's inputs
    rows = [[] for _ in range(4)]  # and output rows

    def run(new_lens, prompts=False):
        x = tokens(sum(new_lens))
        y = s.step(x, new_lens, prompts)
        t = 0
        for r, n in enumerate(new_lens):
            seen[r].append(x[t:t + n])
            rows[r].append(y[t:t + n])
            t += n

    run([37, 150, 5, 0], prompts=True)  # three prompts together; the fourth request waits
    say(f"prompts admitted, cache rows {s.lens.tolist()}")
    for i in range(a.steps):
        # request 3 joins in the middle with a prompt of 90 tokens, in two chunks
        run([1, 1, 1, {3: 50, 4: 40}.get(i, 1 if i > 4 else 0)])
        say(f"step {i}: cache rows {s.lens.tolist()}, {s.free.numel()} blocks free")
    worst = 0.0
    for r in range(4):
        want, got = s.whole(torch.cat(seen[r])), torch.cat(rows[r])
        worst = max(worst, float(((got - want).norm(dim=1) / want.norm(dim=1)).max()))
    say(f"largest relative difference from the whole sequences at once: {worst:.2e}")
    assert lib.qmm_device_status(clear=True) == 0
    return worst


if __name__ == "__main__":
    main()
