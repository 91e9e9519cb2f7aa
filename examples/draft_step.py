"""One attention layer of a speculative decoding step, end to end.

Each sequence of the batch has a committed context in two paged caches that
share a page table: the indexer's keys and the main K/V cache. A draft model
has proposed a tree of tokens per sequence. The step
  1. rotates the drafted tokens' queries to their positions (context + depth),
  2. writes their keys (rotated) and values into the K/V cache, one after
     another behind the context,
  3. asks the indexer for each query's k best committed tokens,
  4. attends to those and to each token's ancestors in the tree.
It then attends to the whole context as well and reports how much of the
attention's weight the selection kept: exp(lse of the selection - lse of all).

    python examples/draft_step.py [--ctx 16384] [--batch 8] [--draft 8] [--k 512] [--fmt fp8]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

FORMATS = {"bf16": 0, "fp8": 1, "fp4": 2}


def draft_tree(n):
    """Parents and depths of n drafted tokens: a chain with a sibling at every
    other level, and the bit rows of their ancestors and themselves."""
    parent = [-1] + [max(0, i - 1 - (i % 2)) for i in range(1, n)]
    depth, row = [0] * n, [1] * n
    for i in range(1, n):
        depth[i] = depth[parent[i]] + 1
        row[i] = row[parent[i]] | (1 << i)
    return depth, row


def run(batch=8, ctx_len=16384, draft=8, k=512, fmt="fp8", heads=64, kv_heads=8, head_dim=128, seed=0):
    """Builds the caches, runs the step, returns a dict of what it computed."""
    import torch

    from dsa_sparse_attention_store_gb300 import PAGE_SIZE, Context, Rope, kv_page_bytes, page_bytes
    dev, f, n = torch.device("cuda"), FORMATS[fmt], draft
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=gen, device=dev).bfloat16()  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)           # noqa: E731

    # handles and buffers a server keeps: the context, a rotary plan, the paged caches, workspaces
    ctx = Context(max_pos=ctx_len + n)
    rope = Rope(ctx, rot_dim=head_dim, max_pos=ctx_len + n)
    pages_each = -(-(ctx_len + n) // PAGE_SIZE)
    pages = batch * pages_each
    table = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).view(batch, pages_each)
    index_cache = torch.zeros(pages * page_bytes(f), dtype=torch.uint8, device=dev)
    kv_cache = torch.zeros(pages * kv_page_bytes(kv_heads, head_dim, f), dtype=torch.uint8, device=dev)
    tokens = batch * n
    topk_ws = torch.empty(ctx.topk_workspace_size(tokens, batch, k, f), dtype=torch.uint8, device=dev)
    attn_ws = torch.empty(ctx.attn_workspace_size(head_dim), dtype=torch.uint8, device=dev)

    # the committed context, as a prefill would have left it
    for b in range(batch):
        pos = torch.arange(ctx_len, dtype=torch.int32, device=dev)
        seq = torch.full_like(pos, b)
        ctx.store(normal(ctx_len, 128), pos, seq, table, index_cache, pages, f)
        ctx.kv_store(normal(ctx_len, kv_heads, head_dim), normal(ctx_len, kv_heads, head_dim), pos, seq, table,
                     kv_cache, pages, f, rope=rope)

    # the drafted tokens
    depth, rows = draft_tree(n)
    place = ints([ctx_len + i for _ in range(batch) for i in range(n)])
    pos = ints([ctx_len + d for _ in range(batch) for d in depth])
    seq = ints([b for b in range(batch) for _ in range(n)])
    words = -(-n // 32)
    signed = lambda v: v - (1 << 32) if v >> 31 else v  # noqa: E731
    mask = ints([[signed((r >> (32 * w)) & 0xFFFFFFFF) for w in range(words)] for _ in range(batch) for r in rows])
    cu_q = ints([b * n for b in range(batch + 1)])
    committed, all_keys = ints([ctx_len] * batch), ints([ctx_len + n] * batch)
    q, key, val = normal(tokens, heads, head_dim) * 2, normal(tokens, kv_heads, head_dim), normal(tokens, kv_heads, head_dim)
    index_q, head_w = normal(tokens, 64, 128), torch.rand((tokens, 64), generator=gen, device=dev) / 8
    chosen = torch.empty((tokens, k), dtype=torch.int32, device=dev)
    score = torch.empty((tokens, k), dtype=torch.float32, device=dev)
    out, lse = torch.empty_like(q), torch.empty((tokens, heads), dtype=torch.float32, device=dev)
    full, full_lse = torch.empty_like(q), torch.empty_like(lse)

    # the step
    ctx.rope_apply(q, pos, rope)
    ctx.kv_store(key, val, place, seq, table, kv_cache, pages, f, rope=rope, rope_pos=pos)
    ctx.topk(index_q, head_w, index_cache, pages, f, table, committed, cu_q, False, k, chosen, score, topk_ws)
    ctx.sparse_attn(q, chosen, kv_cache, pages, f, kv_heads, table, all_keys, cu_q, out, attn_ws, mask=mask, lse=lse)

    # over everything, for comparison
    ctx.tree_attn(q, kv_cache, pages, f, kv_heads, table, all_keys, cu_q, full, attn_ws, mask=mask, lse=full_lse)
    status = ctx.device_status()
    kept = torch.exp(lse - full_lse)
    got = {"status": status, "out": out, "lse": lse, "full": full, "full_lse": full_lse, "kept": kept, "chosen": chosen}
    rope.close()
    ctx.close()
    return got


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--ctx", type=int, default=16384)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--draft", type=int, default=8)
    p.add_argument("--k", type=int, default=512)
    p.add_argument("--fmt", choices=FORMATS, default="fp8")
    a = p.parse_args()
    r = run(a.batch, a.ctx, a.draft, a.k, a.fmt)
    if r["status"]:
        raise SystemExit(f"device status {r['status']}")
    kept = r["kept"].flatten()
    print(f"{a.batch} sequences x {a.draft} drafted tokens over {a.ctx} committed, {a.fmt} caches: {a.k} selected keys keep "
          f"{float(kept.mean()):.3f} of the attention's weight on average ({float(kept.min()):.3f} to {float(kept.max()):.3f})")


if __name__ == "__main__":
    main()
