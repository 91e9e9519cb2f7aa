"""Cases for the operators around the attention over the paged K/V cache: page
tables and slot maps made on the GPU from request lengths, attention of spans
of places (capped scores, distance bias, documents, prefixes, windows), and
attention for batches whose sequences share a long prefix.

Each case names an operator (`op`), its sizes and formats. `run` computes it in
plain torch (32-bit, rounded once at the end) or, where `own` is set, through
the library. Lengths follow from the case alone; contents come from the seed.
"""
import functools
import math

import numpy as np
import torch

own = False

PAGE = 64
BLOCK = 32  # dimensions that share one power-of-two scale in the fp8 and fp4 formats
FMT = {"bf16": 0, "fp8": 1, "fp4": 2}
FP4_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
DEV = "cuda"


# ------------------------------------------------------------------ cases

def _plan(**kw):
    return dict({"op": "plan", "own": 0, "end_every": 0, "pad": 0}, **kw)


def _span(**kw):
    return dict({"op": "span", "kv": 8, "G": 8, "D": 128, "cap": 0.0, "bias": False, "window": 0, "span": "none",
                 "part": 0, "masked": False}, **kw)


def _shared(**kw):
    return dict({"op": "shared", "kv": 8, "G": 8, "D": 128, "cap": 0.0, "bias": False, "window": 0, "masked": False}, **kw)


def listed():
    return [
        # the bookkeeping of one decode step of 64 sequences: launch latency
        _plan(name="plan_decode", B=64, new_min=1, new_max=1, ctx_min=2048, ctx_max=16384),
        # a large server's step: sequences that decode, prompts that go in, some that end, a system
        # prompt's 8 pages that all of them share, a batch padded by 1000 tokens
        _plan(name="plan_large", B=16384, new_min=1, new_max=128, ctx_min=512, ctx_max=8192, own=8, end_every=9, pad=1000),
        # a decode step of a model with capped scores, 64 sequences of ragged lengths
        _span(name="span_decode", B=64, nd=1, ctx_min=2048, ctx_max=16384, fmt="bf16", cap=50.0),
        # the same model's layers that look back 4096 places
        _span(name="span_window_fp8", B=64, nd=1, ctx_min=2048, ctx_max=16384, fmt="fp8", cap=50.0, window=4096),
        # a chunk of a prefill with capped scores behind a committed context
        _span(name="span_chunk", B=1, nd=2048, ctx_min=8192, ctx_max=8192, fmt="bf16", cap=50.0),
        # a prompt of 10498 tokens packed from documents of 512 to 1536 that do not see each other
        _span(name="span_documents", B=1, nd=10498, ctx_min=0, ctx_max=0, fmt="bf16", span="documents", part=1024),
        # short prompts whose first 300 tokens see each other both ways, with a distance bias
        _span(name="span_prefix_fp8", B=5, nd=1000, ctx_min=0, ctx_max=37, kv=4, G=6, D=64, fmt="fp8", bias=True,
              span="prefix", part=300),
        # three new tokens of one short sequence with a distance bias: latency
        _span(name="span_small_fp4", B=1, nd=3, ctx_min=338, ctx_max=338, kv=1, G=16, D=64, fmt="fp4", bias=True),
        # a decode step of 64 sequences behind one prompt of 10498 tokens
        _shared(name="shared_decode", groups=1, size_min=64, size_max=64, nd=1, prefix_min=10498, prefix_max=10498,
                ctx_min=128, ctx_max=1024, fmt="bf16"),
        # four drafted tokens for each sample of eight prompts, capped scores
        _shared(name="shared_samples_fp8", groups=8, size_min=4, size_max=12, nd=4, prefix_min=8192, prefix_max=16384,
                ctx_min=1, ctx_max=2048, fmt="fp8", masked=True, cap=30.0),
        # questions to one book
        _shared(name="shared_long_fp4", groups=1, size_min=32, size_max=32, nd=1, prefix_min=131072, prefix_max=131072,
                ctx_min=16, ctx_max=512, kv=4, G=16, fmt="fp4"),
        # two short sequences behind a short prompt: latency
        _shared(name="shared_small", groups=1, size_min=2, size_max=2, nd=1, prefix_min=704, prefix_max=704, ctx_min=1,
                ctx_max=40, kv=1, G=16, D=64, fmt="bf16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "span", "span", "span", "shared", "shared", "shared"])
    if op == "plan":
        B = _logint(rng, 1, 16384)
        ctx = _logint(rng, 64, 16384)
        while B * ctx > 16384 * 8192:
            ctx //= 2
        new = _logint(rng, 1, max(1, min(22528, 2 ** 20 // B)))
        shared = rng.choice([0, 0, 1, 8])
        low = max(ctx // rng.choice([1, 2, 8]), shared * PAGE)
        return _plan(B=B, new_min=rng.choice([1, new]), new_max=new, ctx_min=low, ctx_max=max(low, ctx), own=shared,
                     end_every=rng.choice([0, 2, 5, 9]), pad=rng.choice([0, 0, 1, 37, 1000]))
    fmt = rng.choice(["bf16", "fp8", "fp4"])
    D = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16]) if rng.random() < 0.8 else rng.choice([32, 64])
    case = {"kv": kv, "G": G, "D": D, "fmt": fmt, "cap": rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]),
            "bias": rng.random() < 0.35, "window": rng.choice([0, 0, 0, 100, 512, 4096])}
    # what a batch may cost: key rows as each sequence has them, and scores
    keys, scores = 2 ** 30 // (kv * D), 2 ** 30 // (kv * G)
    if op == "span":
        nd = _logint(rng, 1, 2048)
        ctx = _logint(rng, 1, 65536)
        while nd * (ctx + nd) > scores:
            nd, ctx = (nd + 1) // 2, (ctx + 1) // 2
        most = min(keys, scores // nd) // (ctx + nd)
        span = rng.choice(["none", "documents", "prefix"])
        case["masked"] = span == "none" and not case["bias"] and nd <= 64 and rng.random() < 0.3
        low = rng.choice([0, ctx // 8, ctx // 2, ctx])
        return _span(B=max(1, min(_logint(rng, 1, 64), most)), nd=nd, ctx_min=low, ctx_max=ctx, span=span,
                     part=0 if span == "none" else _logint(rng, 2, ctx + nd + 1), **case)
    nd = _logint(rng, 1, 64)
    prefix, ctx = _logint(rng, 65, 65536), _logint(rng, 1, 2048)
    size, groups = _logint(rng, 1, 64), _logint(rng, 1, 8)
    while size * groups > 1 and size * groups * (prefix + ctx + nd) > min(keys, scores // nd):
        size, groups = (size + 1) // 2, (groups + 1) // 2
    while nd > 1 and nd * (prefix + ctx + nd) > scores:
        nd //= 2
    case["masked"] = not case["bias"] and rng.random() < 0.5
    return _shared(groups=groups, size_min=rng.choice([1, size]), size_max=size, nd=nd,
                   prefix_min=max(1, prefix // rng.choice([1, 2, 8])), prefix_max=prefix, ctx_min=rng.choice([0, 1, ctx]),
                   ctx_max=ctx, **case)


def _spread(n, lo, hi, steps=(37, 11, 7, 5, 3, 1)):
    """n numbers spread evenly over lo .. hi, in an order that mixes small and large."""
    step = next(s for s in steps if math.gcd(s, n) == 1)
    return [lo + ((i * step) % n) * (hi - lo) // max(1, n - 1) for i in range(n)]


def _plan_lengths(case):
    """Tokens in the cache and tokens to come (-1: the sequence ends)."""
    B, e = case["B"], case["end_every"]
    new = _spread(B, case["new_min"], case["new_max"], (101, 13, 7, 5, 3, 1))
    return _spread(B, case["ctx_min"], case["ctx_max"]), [-1 if e and b % e == e - 1 else n for b, n in enumerate(new)]


def _sizes(case):
    """Sequences of each group."""
    return _spread(case["groups"], case["size_min"], case["size_max"])


def _lengths(case):
    """Committed tokens of each sequence, and how many of them its group shares."""
    if case["op"] == "span":
        return _spread(case["B"], case["ctx_min"], case["ctx_max"]), [0] * case["B"]
    sizes = _sizes(case)
    shared = [p for p, n in zip(_spread(len(sizes), case["prefix_min"], case["prefix_max"]), sizes) for _ in range(n)]
    return [p + c for p, c in zip(shared, _spread(len(shared), case["ctx_min"], case["ctx_max"]))], shared


def _spans(case, c):
    """First place and one past the last place that each new token of a
    sequence with c committed ones sees, by the case's mask alone."""
    nd, part = case["nd"], case["part"]
    place = np.arange(c, c + nd)
    first, last = np.zeros(nd, np.int64), place + 1
    if case["span"] == "documents":  # of part/2 .. 3 part/2 tokens, one after another
        starts, i = [0], 0
        while starts[-1] < c + nd:
            starts.append(starts[-1] + max(1, part * (2 + (i * 7) % 5) // 4))
            i += 1
        first = np.array(starts)[np.searchsorted(starts, place, side="right") - 1]
    elif case["span"] == "prefix":
        last = np.maximum(last, min(part, c + nd))
    return first, last


def _row_bytes(fmt, D):
    return {"bf16": 2 * D, "fp8": D + D // BLOCK, "fp4": D // 2 + D // BLOCK}[fmt]


def _tokens(case):
    return sum(n for n in _plan_lengths(case)[1] if n > 0)


def work(case):
    if case["op"] == "plan":
        old, new = _plan_lengths(case)
        touched = sum((o + n - 1) // PAGE - o // PAGE + 1 for o, n in zip(old, new) if n > 0)
        fresh = sum(-(-(o + n) // PAGE) - -(-o // PAGE) for o, n in zip(old, new) if n > 0)
        ended = sum(-(-o // PAGE) - case["own"] for o, n in zip(old, new) if n < 0)
        return {"bytes": 20 * case["B"] + 12 * (_tokens(case) + case["pad"]) + 4 * (touched + fresh + 2 * ended), "flops": 0}
    ctx, shared = _lengths(case)
    nd, kv, H, D = case["nd"], case["kv"], case["kv"] * case["G"], case["D"]
    keys = pairs = 0
    seen_prefix = {}
    group = [g for g, n in enumerate(_sizes(case)) for _ in range(n)] if case["op"] == "shared" else range(len(ctx))
    for g, c, p in zip(group, ctx, shared):
        first, last = _spans(case, c) if case["op"] == "span" else (np.zeros(nd, np.int64), c + np.arange(nd) + 1)
        if case["window"]:
            first = np.maximum(first, c + np.arange(nd) - case["window"] + 1)
        if case["masked"]:  # its context and itself: what every drafted token sees
            pairs += int(np.maximum(c - first, 0).sum()) + nd
        else:
            pairs += int(np.maximum(last - first, 0).sum())
        lo = int(first.min())
        keys += int(last.max()) - max(lo, p)
        seen_prefix[g] = max(seen_prefix.get(g, 0), p - lo)  # a group's shared places count once
    keys += sum(seen_prefix.values())
    io = len(ctx) * nd * H * (2 * 2 * D + 4)
    return {"bytes": keys * kv * 2 * _row_bytes(case["fmt"], D) + io, "flops": pairs * H * D * 4}


# ------------------------------------------------------------------ formats

def _fp4_edges(device):
    """Upper edges of the codes 0..6: a value above edge i has a code above i;
    on the edge it takes the even code."""
    e = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float32, device=device)
    below = torch.nextafter(e, torch.zeros_like(e))
    return torch.where(torch.arange(7, device=device) % 2 == 1, below, e)


def _quantise(y, fmt):
    """fp32 [..., D] -> (codes uint8 [..., code bytes], scales uint8 [..., D/32] or None)."""
    if fmt == "bf16":
        return y.to(torch.bfloat16).view(torch.uint8), None
    blocks = y.reshape(*y.shape[:-1], -1, BLOCK)
    m, e = torch.frexp(blocks.abs().amax(-1))
    e = (e - 9 + (m > 0.875)).clamp(-117, 119) if fmt == "fp8" else (e - 3 + (m > 0.75)).clamp(-125, 125)
    x = torch.ldexp(blocks, -e.unsqueeze(-1)).reshape(y.shape)
    scales = (e + 127).to(torch.uint8)
    if fmt == "fp8":
        return x.to(torch.float8_e4m3fn).view(torch.uint8), scales
    code = torch.bucketize(x.abs(), _fp4_edges(y.device)).to(torch.uint8)
    code = torch.where(torch.signbit(x), code + 8, code)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _dequantise(codes, scales, fmt, dtype):
    if fmt == "bf16":
        return codes.view(torch.bfloat16).to(dtype)
    if fmt == "fp8":
        x = codes.view(torch.float8_e4m3fn).to(dtype)
    else:
        table = torch.tensor(FP4_VALUES + [-v for v in FP4_VALUES], dtype=dtype, device=codes.device)
        x = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    blocks = x.reshape(*x.shape[:-1], -1, BLOCK)
    return torch.ldexp(blocks, scales.to(torch.int32).unsqueeze(-1) - 127).reshape(x.shape)


def _fields(cache, case):
    """Views of a cache [pages, kv, bytes] as K and V codes [pages, kv, 64, code
    bytes] and scales [pages, kv, 64, D/32] (None for bf16)."""
    D, fmt = case["D"], case["fmt"]
    cb = {"bf16": 2 * D, "fp8": D, "fp4": D // 2}[fmt]
    sb = 0 if fmt == "bf16" else D // BLOCK
    cut = lambda at, n: cache[:, :, at:at + PAGE * n].unflatten(2, (PAGE, n))  # noqa: E731
    kc, vc = cut(0, cb), cut(PAGE * cb, cb)
    if not sb:
        return kc, None, vc, None
    return kc, cut(2 * PAGE * cb, sb), vc, cut(2 * PAGE * cb + PAGE * sb, sb)


# ------------------------------------------------------------------ states

@functools.lru_cache(maxsize=None)
def _context():
    from dsa_sparse_attention_store_gb300 import Context
    return Context(max_pos=64)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _paging(lens, shared, gen):
    """A page table over randomly placed pages for sequences of these lengths;
    neighbours that share a prefix (`shared`: its whole pages, by group) point
    to the same ones. shared: list of (first sequence, sequences, pages)."""
    pages = [-(-n // PAGE) for n in lens]
    total = sum(pages) + 3
    order = torch.randperm(total, generator=gen, device=DEV)[:sum(pages)].to(torch.int32)
    table = torch.zeros((len(lens), max(pages)), dtype=torch.int32, device=DEV)
    table[torch.arange(max(pages), device=DEV)[None, :] < _int(pages)[:, None]] = order
    for at, n, p in shared:
        table[at:at + n, :p] = table[at, :p].clone()
    return table, total


def _tree(B, nd, gen):
    """Random trees of drafted tokens as bit rows: bit j of row i is set where
    token j is token i or one of its ancestors."""
    u = torch.rand((B, nd), generator=gen, device=DEV)
    at = torch.arange(nd, device=DEV)
    # the parent of token i is one of the tokens before it, mostly a recent one; token 0 is the root
    parent = (at[None, :] - 1 - (u * u * at).floor().long()).clamp(min=0)
    seen = torch.eye(nd, dtype=torch.bool, device=DEV).repeat(B, 1, 1)
    for i in range(1, nd):
        seen[:, i] |= seen[torch.arange(B, device=DEV), parent[:, i]]
    words = -(-nd // 32)
    bits = torch.zeros((B, nd, words * 32), dtype=torch.int64, device=DEV)
    bits[..., :nd] = seen
    value = (bits.view(B, nd, words, 32) << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(value >= 2 ** 31, value - 2 ** 32, value).to(torch.int32).view(B * nd, words)


def _prepare_plan(case, gen):
    old, new = _plan_lengths(case)
    B, keep = case["B"], case["own"]
    P0 = [-(-o // PAGE) for o in old]
    need = sum(-(-(o + n) // PAGE) - p for o, n, p in zip(old, new, P0) if n > 0)
    width = max(-(-(o + max(n, 0)) // PAGE) for o, n in zip(old, new))
    free = need + 5
    total = sum(P0) + free
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None, :] < _int(P0)[:, None]] = order[:sum(P0)]
    table[:, :keep] = table[0, :keep].clone()  # of the first sequence
    stack = torch.full((total,), -1, dtype=torch.int32, device=DEV)
    stack[:free] = order[sum(P0):]
    T = _tokens(case) + case["pad"]
    empty = lambda *n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    s = {"case": case, "pages": total, "old": _int(old), "new": _int(new), "table": table, "stack": stack, "count": _int([free]),
         "left": empty(1), "lens": empty(B), "cu_q": empty(B + 1), "seq": empty(T), "pos": empty(T), "slot": empty(T),
         "own_from": _int([0] + [keep] * (B - 1)) if keep else None,
         # what the host knows of the step: new pages, pages of sequences that end
         "fresh": need, "ended": sum(p - (keep if b else 0) for b, (p, n) in enumerate(zip(P0, new)) if n < 0)}
    if own:
        s["ctx"] = _context()
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "plan":
        return _prepare_plan(case, gen)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    kv, D, nd = case["kv"], case["D"], case["nd"]
    ctx, shared = _lengths(case)
    B, H = len(ctx), kv * case["G"]
    s = {"case": case}
    groups, at = [], 0
    if case["op"] == "shared":
        for n in _sizes(case):
            groups.append((at, n, shared[at] // PAGE))
            at += n
        s["cu_groups"] = _int([g[0] for g in groups] + [B])
        s["shared"] = _int([shared[g[0]] for g in groups])
    s["table"], s["pages"] = _paging([c + nd for c in ctx], groups, gen)
    s["lens"] = _int([c + nd for c in ctx])
    s["cu_q"] = _int([b * nd for b in range(B + 1)])
    row = 2 * PAGE * _row_bytes(case["fmt"], D)  # bytes of one kv head's part of a page
    s["cache"] = torch.empty((s["pages"], kv, row), dtype=torch.uint8, device=DEV)
    kc, ks, vc, vs = _fields(s["cache"], case)
    for i in range(0, s["pages"], 1024):  # a part at a time: the 32-bit values of a long context are large
        n = min(1024, s["pages"] - i)
        for codes, scales in ((kc, ks), (vc, vs)):
            c, e = _quantise(normal(n, kv, PAGE, D), case["fmt"])
            codes[i:i + n] = c
            if e is not None:
                scales[i:i + n] = e
    # scores of a standard deviation of 4: the best of them feel a cap of 20 to 50
    s["q"] = (normal(B * nd, H, D) * 4.0).to(torch.bfloat16)
    s["mask"] = _tree(B, nd, gen) if case["masked"] else None
    s["slopes"] = None
    if case["bias"]:  # halving over the heads, as such models have them
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32, device=DEV) / H)
    s["first"] = s["last"] = None
    if case["op"] == "span" and case["span"] != "none":
        spans = [_spans(case, c) for c in ctx]
        which = 0 if case["span"] == "documents" else 1
        s["first" if which == 0 else "last"] = _int(np.concatenate([x[which] for x in spans]).tolist())
    if own:
        s["ctx"] = _context()
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B * nd, H), dtype=torch.float32, device=DEV)
        if case["op"] == "span":
            size = s["ctx"].span_attn_workspace_size(B * nd, B, H, kv, D)
        else:
            size = s["ctx"].shared_attn_workspace_size(B * nd, B, len(groups), H, kv, D)
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if s["case"]["op"] == "plan":
        return (_run_own_plan if own else _run_plain_plan)(s)
    return (_run_own if own else _run_plain)(s)


def _plan_outputs(s):
    return {k: s[k] for k in ("table", "stack", "left", "lens", "cu_q", "seq", "pos", "slot")}


def _run_own_plan(s):
    s["ctx"].batch_plan(s["old"], s["new"], s["table"], s["pages"], s["stack"], s["count"], s["left"], s["lens"], s["cu_q"],
                        s["seq"], s["pos"], s["slot"], own_from=s["own_from"])
    return _plan_outputs(s)


def _run_own(s):
    case, ctx = s["case"], s["ctx"]
    more = {"mask": s["mask"], "lse": s["lse"], "cap": case["cap"], "slopes": s["slopes"], "window": case["window"],
            "first": s["first"], "last": s["last"]}
    args = (s["q"], s["cache"].view(-1), s["pages"], FMT[case["fmt"]], case["kv"], s["table"], s["lens"], s["cu_q"], s["out"],
            s["ws"])
    if case["op"] == "span":
        ctx.span_attn(*args, **more)
    else:
        ctx.shared_attn(*args, s["cu_groups"], s["shared"], **more)
    return {"out": s["out"], "lse": s["lse"]}


def _run_plain_plan(s):
    """Pages that a sequence needs come from the end of the list (free pages,
    then the pages of sequences that end); what is left of it is free."""
    old, new, table, stack = s["old"].long(), s["new"].long(), s["table"], s["stack"]
    B, T, count = old.shape[0], s["seq"].shape[0], s["count"].long()
    keep = torch.zeros_like(old) if s["own_from"] is None else s["own_from"].long()
    ends = new < 0
    lens = torch.where(ends, 0, old + new)
    P0, P1 = (old + PAGE - 1) // PAGE, (lens + PAGE - 1) // PAGE
    zero = torch.zeros_like(old)
    fresh, ended = torch.where(ends, zero, P1 - P0), torch.where(ends, (P0 - keep).clamp(min=0), zero)
    A, R = s["fresh"], s["ended"]
    b = torch.arange(B, device=DEV)
    before = lambda x: torch.cumsum(x, 0) - x  # noqa: E731
    rb = torch.repeat_interleave(b, ended, output_size=R)
    freed = table[rb, keep[rb] + torch.arange(R, device=DEV) - before(ended)[rb]].long()
    ab = torch.repeat_interleave(b, fresh, output_size=A)
    i = torch.arange(A, device=DEV)
    v = count + R - 1 - i
    page = stack[v.clamp(min=0).minimum(count - 1)].long()
    if R:
        page = torch.where(v >= count, freed[(v - count).clamp(min=0)], page)
    table[ab, P0[ab] + i - before(fresh)[ab]] = page.to(torch.int32)
    if R > A:
        stack[count + torch.arange(R - A, device=DEV)] = freed[:R - A].to(torch.int32)
    n = torch.where(ends, zero, new)
    s["left"].copy_(count + R - A)
    s["lens"].copy_(lens)
    s["cu_q"][0] = 0
    s["cu_q"][1:] = torch.cumsum(n, 0)
    total = T - s["case"]["pad"]
    tb = torch.repeat_interleave(b, n, output_size=total)
    pos = old[tb] + torch.arange(total, device=DEV) - before(n)[tb]
    for out, x in (("seq", tb), ("pos", pos), ("slot", table[tb, pos // PAGE].long() * PAGE + pos % PAGE)):
        s[out][:total] = x.to(torch.int32)
        s[out][total:] = -1
    return _plan_outputs(s)


def _run_plain(s):
    case = s["case"]
    kc, ks, vc, vs = _fields(s["cache"], case)
    fmt, nd, kv, G, D = case["fmt"], case["nd"], case["kv"], case["G"], case["D"]
    lens = s["lens"].long()
    B, L = lens.shape[0], s["table"].shape[1] * PAGE
    ctx = lens - nd
    pos = torch.arange(L, device=DEV)
    place = ctx[:, None] + torch.arange(nd, device=DEV)
    last = s["last"].long().view(B, nd) if s["last"] is not None else lens[:, None] if case["masked"] else place + 1
    see = (pos < last[..., None].expand(B, nd, 1)) & (pos < lens[:, None, None])
    if s["first"] is not None:
        see &= pos >= s["first"].long().view(B, nd, 1)
    if case["window"]:
        see &= pos > place[..., None] - case["window"]
    if s["mask"] is not None:
        bit = (s["mask"].view(B, nd, -1, 1) >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        j = (pos - ctx[:, None]).clamp(0, nd - 1)[:, None, :].expand(-1, nd, -1)
        see &= (pos < ctx[:, None])[:, None, :] | bit.flatten(2)[..., :nd].bool().gather(2, j)
    see = see[:, :, None, :].expand(-1, -1, G, -1).reshape(B, nd * G, L)
    page, off = s["table"].long()[:, pos // PAGE], pos % PAGE
    q = s["q"].view(B, nd, kv, G, D)
    out = torch.empty((B, nd, kv, G, D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((B, nd, kv, G), dtype=torch.float32, device=DEV)
    for h in range(kv):
        field = lambda x: None if x is None else x[page, h, off]  # noqa: E731,B023
        k = _dequantise(field(kc), field(ks), fmt, torch.float32)
        score = torch.matmul(q[:, :, h].reshape(B, nd * G, D).float(), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
        del k
        if case["cap"]:
            score = score.div_(case["cap"]).tanh_().mul_(case["cap"])
        if s["slopes"] is not None:
            far = (place[..., None] - pos).abs().float()
            score = score.view(B, nd, G, L).sub_(far[:, :, None, :] * s["slopes"][h * G:(h + 1) * G, None]).view(B, nd * G, L)
        score = score.masked_fill_(~see, -math.inf)
        top = score.amax(-1, keepdim=True)
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        p = score.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        v = _dequantise(field(vc), field(vs), fmt, torch.float32)
        o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
        out[:, :, h] = o.view(B, nd, G, D).to(torch.bfloat16)
        lse[:, :, h] = (top + torch.log(total)).view(B, nd, G)
        del p, score, v
    return {"out": out.view(B * nd, kv * G, D), "lse": lse.view(B * nd, kv * G)}


# ------------------------------------------------------------------ the definition, on the host or in 64 bits

def _exact_plan(case, s):
    """Sequence by sequence, with a list of pages that grows and shrinks."""
    old, new = _plan_lengths(case)
    table, stack = s["table"].cpu().numpy().copy(), s["stack"].cpu().numpy().copy()
    count = int(s["count"])
    keep = [0] * case["B"] if s["own_from"] is None else s["own_from"].tolist()
    pool = stack[:count].tolist()
    for b, (o, n) in enumerate(zip(old, new)):
        if n < 0:
            pool += table[b, keep[b]:-(-o // PAGE)].tolist()
    T = s["seq"].shape[0]
    seq, pos, slot = (np.full(T, -1, np.int32) for _ in range(3))
    lens, cu_q = [], [0]
    for b, (o, n) in enumerate(zip(old, new)):
        m = max(n, 0)
        if n >= 0:
            for p in range(-(-o // PAGE), -(-(o + n) // PAGE)):
                table[b, p] = pool.pop()
            at, where = cu_q[-1], np.arange(o, o + m)
            seq[at:at + m], pos[at:at + m] = b, where
            slot[at:at + m] = table[b, where // PAGE] * PAGE + where % PAGE
        lens.append(o + n if n >= 0 else 0)
        cu_q.append(cu_q[-1] + m)
    if len(pool) > count:
        stack[count:len(pool)] = pool[count:]
    up = lambda x: torch.as_tensor(np.asarray(x, np.int32), device=DEV)  # noqa: E731
    return {"table": up(table), "stack": up(stack), "left": up([len(pool)]), "lens": up(lens), "cu_q": up(cu_q),
            "seq": up(seq), "pos": up(pos), "slot": up(slot)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(case, s)
    nd, kv, G, D = case["nd"], case["kv"], case["G"], case["D"]
    ctx, _ = _lengths(case)
    out = torch.zeros((len(ctx) * nd, kv * G, D), dtype=torch.float64, device=DEV)
    lse = torch.full((len(ctx) * nd, kv * G), -math.inf, dtype=torch.float64, device=DEV)
    fields = _fields(s["cache"], case)
    slopes = None if s["slopes"] is None else s["slopes"].double()
    words = None if s["mask"] is None else s["mask"].cpu().numpy().astype(np.uint32)
    for b, c in enumerate(ctx):
        first, last = _spans(case, c) if case["op"] == "span" else (np.zeros(nd, np.int64), c + np.arange(nd) + 1)
        if case["masked"]:
            last = np.full(nd, c + nd)
        if case["window"]:
            first = np.maximum(first, c + np.arange(nd) - case["window"] + 1)
        bits = None
        if words is not None:
            bits = np.unpackbits(np.ascontiguousarray(words[b * nd:(b + 1) * nd]).view(np.uint8), axis=1, bitorder="little")
        for i0 in range(0, nd, 512):  # some queries at a time, over the places that one of them sees
            i1 = min(nd, i0 + 512)
            lo, hi = int(first[i0:i1].min()), int(last[i0:i1].max())
            where = torch.arange(lo, hi, device=DEV)
            see = (np.arange(lo, hi) >= first[i0:i1, None]) & (np.arange(lo, hi) < last[i0:i1, None])
            if bits is not None:
                drafted = np.arange(lo, hi) - c
                see &= np.where(drafted < 0, True, bits[i0:i1][:, np.clip(drafted, 0, nd - 1)].astype(bool))
            see = torch.from_numpy(see).to(DEV).repeat_interleave(G, 0)
            slot = s["table"][b, where // PAGE].long() * PAGE + where % PAGE
            far = (torch.arange(c + i0, c + i1, device=DEV)[:, None] - where).abs().double()
            rows = slice(b * nd + i0, b * nd + i1)
            for h in range(kv):
                flat = [None if x is None else x[:, h].flatten(0, 1)[slot] for x in fields]
                k, v = (_dequantise(flat[j], flat[j + 1], case["fmt"], torch.float64) for j in (0, 2))
                heads = slice(h * G, (h + 1) * G)
                z = s["q"][rows, heads].double().reshape((i1 - i0) * G, D) @ k.T / math.sqrt(D)
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if slopes is not None:
                    z = z - (slopes[heads][None, :, None] * far[:, None, :]).reshape(z.shape)
                z = z.masked_fill(~see, -math.inf)
                total = torch.logsumexp(z, -1)
                w = torch.exp(z - torch.where(torch.isfinite(total), total, torch.zeros_like(total))[:, None])
                out[rows, heads] = (w @ v).view(i1 - i0, G, D)
                lse[rows, heads] = total.view(i1 - i0, G)
    return {"out": out, "lse": lse}
