"""One attention layer of a server that draws several samples behind a prompt.

A pool of pages serves every sequence. The server's steps are
  1. the prompt goes in: batch_plan takes its pages and says where its tokens
     go, kv_store writes their keys (rotated) and values there, span_attn attends
     with capped scores, each token over its own document of the prompt;
  2. the samples fork: their rows of the page table begin with the prompt's whole
     pages, the rest of its tokens goes into a page of each one's own;
  3. decode steps: batch_plan gives each sample a place (and, now and then, a
     page), kv_store writes, shared_attn reads the prompt once for all of them;
  4. the samples end, and their pages come back.
The decode steps are also made with span_attn, which reads the prompt once a
sample, and the largest difference is reported.

    python examples/shared_prompt.py [--prompt 4509] [--document 700] [--samples 8] [--steps 4] [--fmt bf16]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

FORMATS = {"bf16": 0, "fp8": 1, "fp4": 2}


def run(prompt=4509, samples=8, steps=4, fmt="bf16", heads=32, kv_heads=4, head_dim=128, cap=50.0, seed=0, document=700):
    """Runs the steps, returns a dict of what they computed. document: tokens of
    each of the prompt's documents."""
    import torch

    from dsa_sparse_attention_store_gb300 import PAGE_SIZE, Context, Rope, kv_page_bytes
    dev, f = torch.device("cuda"), FORMATS[fmt]
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=gen, device=dev).bfloat16()  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)           # noqa: E731
    empty = lambda *s: torch.empty(s, dtype=torch.int32, device=dev)          # noqa: E731

    # what a server keeps: the context, a rotary plan, the cache, the pool and the rows of B sequences
    B, width = samples + 1, -(-(prompt + steps) // PAGE_SIZE)
    pages = -(-prompt // PAGE_SIZE) + samples * (width - prompt // PAGE_SIZE)  # the prompt's, and each sample's own behind its whole ones
    ctx = Context(max_pos=64)
    rope = Rope(ctx, rot_dim=head_dim, max_pos=prompt + steps)
    cache = torch.zeros(pages * kv_page_bytes(kv_heads, head_dim, f), dtype=torch.uint8, device=dev)
    pool, count, left = torch.randperm(pages, generator=gen, device=dev).to(torch.int32), ints([pages]), empty(1)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    old, lens, cu_q = ints([0] * B), empty(B), empty(B + 1)

    def step(new, tokens, own_from=None):
        """Places of the step's new tokens; then what was taken is what there is."""
        seq, place, slot = empty(tokens), empty(tokens), empty(tokens)
        ctx.batch_plan(old, ints(new), table, pages, pool, count, left, lens, cu_q, seq, place, slot, own_from=own_from)
        count.copy_(left)
        old.copy_(lens)
        return seq, place

    def write(seq, place, k, v):
        ctx.kv_store(k, v, place, seq, table, cache, pages, f, rope=rope)

    got = {}
    # 1. the prompt is sequence 0, packed from documents
    seq, place = step([prompt] + [0] * samples, prompt)
    k, v, q = normal(prompt, kv_heads, head_dim), normal(prompt, kv_heads, head_dim), normal(prompt, heads, head_dim) * 3
    write(seq, place, k, v)
    ctx.rope_apply(q, place, rope)
    out, lse = torch.empty_like(q), torch.empty((prompt, heads), device=dev)
    ws = torch.empty(ctx.span_attn_workspace_size(prompt, B, heads, kv_heads, head_dim), dtype=torch.uint8, device=dev)
    ctx.span_attn(q, cache, pages, f, kv_heads, table, lens, cu_q, out, ws, lse=lse, cap=cap, first=place - place % document)
    got.update(prompt_q=q.clone(), prompt_out=out, prompt_lse=lse)

    # 2. the samples point to the prompt's whole pages; its last tokens they have for themselves
    whole = prompt // PAGE_SIZE
    table[1:, :whole] = table[0, :whole]
    old[1:] = whole * PAGE_SIZE
    own_from = ints([0] + [whole] * samples)
    rest = prompt - whole * PAGE_SIZE
    if rest:
        seq, place = step([0] + [rest] * samples, rest * samples)
        write(seq, place, k[whole * PAGE_SIZE:].repeat(samples, 1, 1), v[whole * PAGE_SIZE:].repeat(samples, 1, 1))

    # 3. decode; the group is the samples, behind the prompt
    cu_groups, shared = ints([1, B]), ints([prompt])
    ws = torch.empty(ctx.shared_attn_workspace_size(samples, B, 1, heads, kv_heads, head_dim), dtype=torch.uint8, device=dev)
    got["steps"] = []
    for _ in range(steps):
        seq, place = step([0] + [1] * samples, samples)
        k, v, q = normal(samples, kv_heads, head_dim), normal(samples, kv_heads, head_dim), normal(samples, heads, head_dim) * 3
        write(seq, place, k, v)
        ctx.rope_apply(q, place, rope)
        out, lse = torch.empty_like(q), torch.empty((samples, heads), device=dev)
        ctx.shared_attn(q, cache, pages, f, kv_heads, table, lens, cu_q, out, ws, cu_groups, shared, lse=lse, cap=cap)
        alone, alone_lse = torch.empty_like(q), torch.empty_like(lse)
        ctx.span_attn(q, cache, pages, f, kv_heads, table, lens, cu_q, alone, ws, lse=alone_lse, cap=cap)
        got["steps"].append(dict(q=q, out=out, lse=lse, alone=alone, alone_lse=alone_lse, lens=lens.clone()))

    # 4. the samples end; the pages that are theirs come back
    got.update(table=table.clone(), cache=cache.clone(), pages=pages, before_end=int(count))
    step([0] + [-1] * samples, 0, own_from=own_from)
    got.update(after_end=int(count), pool=pool.clone(), rows=table, status=ctx.device_status())
    rope.close()
    ctx.close()
    return got


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--prompt", type=int, default=4509)
    p.add_argument("--document", type=int, default=700)
    p.add_argument("--samples", type=int, default=8)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--fmt", choices=FORMATS, default="bf16")
    a = p.parse_args()
    r = run(a.prompt, a.samples, a.steps, a.fmt, document=a.document)
    if r["status"]:
        raise SystemExit(f"device status {r['status']}")
    far = max(float((s["lse"] - s["alone_lse"]).abs().max()) for s in r["steps"])
    print(f"{a.samples} samples of {a.steps} steps behind {a.prompt} tokens, {a.fmt}: lse with the prompt read once is within {far:.1e} of "
          f"lse with it read for each; {r['after_end'] - r['before_end']} pages came back")


if __name__ == "__main__":
    main()
