"""A batch of sequences decoded through one attention layer with random weights.

The prompt's keys are rotated and stored in a paged 8-bit cache in one call, then every step projects one
token a sequence, rotates its query, stores its key and value and attends over the cache.  Sequences have
lengths of their own and take pages from one pool as they grow.

    python examples/decode.py [--batch 8] [--heads 32] [--kv-heads 8] [--dim 128] [--prompt 1000] [--steps 32]
                              [--cache e4m3|int8|bf16] [--window 0] [--check]

--check compares every step with the same layer computed plainly in 64 bits from the values the cache holds.
"""

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layout_remapping_copy_amd as lr  # noqa: E402

TYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16}


class Pool:
    """Pages of a cache (slots first, heads next to each other) and each sequence's list of them."""

    def __init__(self, kind, batch, most, kv_heads, dim, page, device):
        self.page, self.width = page, -(-most // page)
        pages = batch * self.width
        k, v = (torch.zeros(pages * page * kv_heads * dim, dtype=torch.uint8 if kind == "e4m3" else TYPES[kind], device=device)
                for _ in range(2))
        layout = f"({dim},{kv_heads},{page},{pages}):(1,{dim},{kv_heads * dim},{page * kv_heads * dim})"
        scales = (None, None, None)
        if kind != "bf16":
            scales = (*(torch.zeros(pages * page * kv_heads, device=device) for _ in range(2)),
                      f"({kv_heads},{page},{pages}):(1,{kv_heads},{page * kv_heads})")
        self.cache = lr.PagedCache(k, layout, v, layout, *scales)
        self.table = torch.full((batch, self.width), -1, dtype=torch.int32, device=device)
        self.free = torch.randperm(pages).tolist()
        self.held = [0] * batch

    def grow(self, lens):
        """Pages for the first lens[b] tokens of every sequence b."""
        for b, n in enumerate(lens):
            while self.held[b] * self.page < n:
                self.table[b, self.held[b]] = self.free.pop()
                self.held[b] += 1

    def slots(self, sequence, position):
        """The cache's slot of each token (int64 tensors of the same length)."""
        return self.table.long()[sequence, position // self.page] * self.page + position % self.page


def run(batch=8, heads=32, kv_heads=8, dim=128, prompt=1000, steps=32, cache="e4m3", window=0, page=16, check=False,
        device="cuda", seed=0):
    """Returns (seconds a step, the last step's outputs, the worst error of a step over its tolerance with check)."""
    torch.manual_seed(seed)
    dtype, width = torch.bfloat16, heads * dim
    wq, wk, wv, wo = (torch.randn(m, n, device=device, dtype=dtype) / math.sqrt(m)
                      for m, n in ((width, width), (width, kv_heads * dim), (width, kv_heads * dim), (width, width)))
    lens = [max(1, prompt - 37 * b % prompt) for b in range(batch)]
    pool = Pool(cache, batch, max(lens) + steps, kv_heads, dim, page, device)
    table = lr.rope_table(dim, base=500000.0, device=device)
    # the prompt: all tokens of all sequences in one call
    pool.grow(lens)
    sequence = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).to(device)
    position = torch.cat([torch.arange(n) for n in lens]).to(device)
    x = torch.randn(len(sequence), width, device=device, dtype=dtype)
    Lkv = lr.Layout(f"({dim},{kv_heads},{len(sequence)}):(1,{dim},{kv_heads * dim})")
    lr.cache_write(pool.cache, x @ wk, Lkv, x @ wv, Lkv, pool.slots(sequence, position), table=table, positions=position)
    # the steps
    Lq = lr.Layout(f"({dim},{heads},{batch}):(1,{dim},{width})")
    Lkv = lr.Layout(f"({dim},{kv_heads},{batch}):(1,{dim},{kv_heads * dim})")
    plan = lr.paged_attention_plan(Lq, pool.cache, Lq, pool.width, dtype, window=window)
    workspace = torch.empty(plan["workspace_bytes"], dtype=torch.uint8, device=device)
    every, out, worst, spent = torch.arange(batch, device=device), None, 0.0, 0.0
    x = torch.randn(batch, width, device=device, dtype=dtype)
    for _ in range(steps):
        position = torch.tensor(lens, device=device)
        lens = [n + 1 for n in lens]
        pool.grow(lens)
        slots, seen = pool.slots(every, position), torch.tensor(lens, dtype=torch.int32, device=device)
        torch.cuda.synchronize()
        start = time.perf_counter()
        q, k, v = x @ wq, x @ wk, x @ wv
        lr.rope(q, Lq, q, Lq, position, table)
        lr.cache_write(pool.cache, k, Lkv, v, Lkv, slots, table=table, positions=position)
        out = lr.paged_attention(q, Lq, pool.cache, pool.table, seen, torch.empty_like(q), Lq, window=window,
                                 workspace=workspace)
        x = torch.nn.functional.layer_norm((x + out @ wo).float(), (width,)).to(dtype)
        torch.cuda.synchronize()
        spent += time.perf_counter() - start
        if check:
            worst = max(worst, error(pool, q, out, lens, heads, kv_heads, dim, window))
    return spent / steps, out, worst


def error(pool, q, out, lens, heads, kv_heads, dim, window):
    """The largest error of out over half a step of bf16 in its size and the size of the values."""
    worst = 0.0
    for b, n in enumerate(lens):
        at = torch.arange(max(0, n - window) if window else 0, n, device=q.device)
        k, v = (torch.empty(len(at), kv_heads, dim, device=q.device, dtype=torch.float32) for _ in range(2))
        slots = pool.slots(torch.full_like(at, b), at)
        L = f"({dim},{kv_heads},{len(at)}):(1,{dim},{kv_heads * dim})"
        if pool.cache.k_scale is None:
            k, v = k.to(q.dtype), v.to(q.dtype)
        lr.cache_read(pool.cache, slots, k, L, v, L)
        k, v = (z.double().cpu().repeat_interleave(heads // kv_heads, 1).transpose(0, 1) for z in (k, v))
        w = torch.softmax((k @ q[b].view(heads, dim, 1).double().cpu()).squeeze(-1) / math.sqrt(dim), -1)
        want = (w.unsqueeze(1) @ v).squeeze(1)
        size = (w.unsqueeze(1) @ v.abs()).squeeze(1)
        off = (out[b].view(heads, dim).double().cpu() - want).abs()
        worst = max(worst, float((off / (2.0 ** -8 * want.abs() + 2.0 ** -12 * size)).max()))
    return worst


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("batch", 8), ("heads", 32), ("kv-heads", 8), ("dim", 128), ("prompt", 1000), ("steps", 32), ("window", 0)):
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--cache", choices=sorted(TYPES), default="e4m3")
    p.add_argument("--check", action="store_true")
    a = p.parse_args()
    seconds, _, worst = run(a.batch, a.heads, a.kv_heads, a.dim, a.prompt, a.steps, a.cache, a.window, check=a.check)
    print(f"{a.batch} sequences, {a.steps} steps: {seconds * 1e6:.0f} us a step, {a.batch / seconds:.0f} tokens/s")
    if a.check:
        print(f"largest error of a step: {worst:.2f} of its tolerance")
        if not worst <= 1:
            sys.exit(1)


if __name__ == "__main__":
    main()
