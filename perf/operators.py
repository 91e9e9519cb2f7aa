"""Cases for the operators that follow the indexer: rotary positions, the
quantised K/V cache, attention of drafted tokens over the cache and attention
over the indexer's selection.

Each case names an operator (`op`), its sizes and formats. `run` computes it in
plain torch (32-bit, rounded once at the end) or, where `own` is set, through
the library. The context lengths of a batch follow from the case alone (spread
between `ctx_min` and `ctx_max`); contents come from the seed.
"""
import functools
import math

import numpy as np
import torch

own = False

PAGE = 64
BLOCK = 32  # dimensions that share one power-of-two scale in the fp8 and fp4 formats
FMT = {"bf16": 0, "fp8": 1, "fp4": 2}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP4_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # rotating the 64 query heads of one decode step of 64 sequences: launch latency
        {"name": "rope_decode", "op": "rope", "T": 64, "H": 64, "D": 128, "rot": 128, "start": 0,
         "layout": "half", "scaling": "none", "factor": 1.0, "dtype": "bf16", "inverse": False,
         "max_pos": 16384},
        # the queries of a 22528-token prefill, the last 64 dimensions rotated,
        # positions scaled for a long context
        {"name": "rope_prefill", "op": "rope", "T": 22528, "H": 64, "D": 128, "rot": 64, "start": 64,
         "layout": "interleaved", "scaling": "by_parts", "factor": 4.0, "dtype": "bf16",
         "inverse": False, "max_pos": 131072},
        # one decode step's keys and values written (keys rotated) and read back: latency
        {"name": "kv_decode_fp8", "op": "kv", "T": 64, "B": 64, "kv": 8, "D": 128, "fmt": "fp8",
         "rot": 128, "start": 0, "layout": "half", "ctx": 10498},
        # a 22528-token prefill written and read back
        {"name": "kv_prefill_fp4", "op": "kv", "T": 22528, "B": 1, "kv": 8, "D": 128, "fmt": "fp4",
         "rot": 64, "start": 0, "layout": "interleaved", "ctx": 0},
        # a single-token decode step, 64 sequences of ragged lengths
        {"name": "tree_decode", "op": "tree", "B": 64, "nd": 1, "ctx_min": 2048, "ctx_max": 16384,
         "kv": 8, "G": 8, "D": 128, "fmt": "bf16", "masked": True},
        # eight drafted tokens over long contexts
        {"name": "tree_long_fp8", "op": "tree", "B": 8, "nd": 8, "ctx_min": 131072, "ctx_max": 131072,
         "kv": 4, "G": 16, "D": 128, "fmt": "fp8", "masked": True},
        # wide trees: 64 drafted tokens for each of 16 sequences
        {"name": "tree_wide", "op": "tree", "B": 16, "nd": 64, "ctx_min": 4509, "ctx_max": 10498,
         "kv": 8, "G": 8, "D": 128, "fmt": "bf16", "masked": True},
        # one short sequence, a small tree: latency
        {"name": "tree_small_fp4", "op": "tree", "B": 1, "nd": 5, "ctx_min": 338, "ctx_max": 338,
         "kv": 1, "G": 16, "D": 64, "fmt": "fp4", "masked": True},
        # a chunk of a prefill (a chain of tokens, no mask) behind a committed context
        {"name": "tree_chunk", "op": "tree", "B": 1, "nd": 2048, "ctx_min": 8192, "ctx_max": 8192,
         "kv": 8, "G": 8, "D": 128, "fmt": "bf16", "masked": False},
        # decode over the 512 selected tokens, one shared kv head
        {"name": "sparse_decode_fp8", "op": "sparse", "B": 64, "nd": 1, "ctx_min": 2048,
         "ctx_max": 16384, "k": 512, "kv": 1, "G": 64, "D": 128, "fmt": "fp8", "masked": False},
        # 2048 queries of a prefill, each over its own selection
        {"name": "sparse_prefill", "op": "sparse", "B": 1, "nd": 2048, "ctx_min": 20480,
         "ctx_max": 20480, "k": 512, "kv": 8, "G": 8, "D": 128, "fmt": "bf16", "masked": False},
        # drafted tokens over long contexts: the selection and the tree's own tokens
        {"name": "sparse_long_fp4", "op": "sparse", "B": 8, "nd": 8, "ctx_min": 131072,
         "ctx_max": 131072, "k": 1024, "kv": 2, "G": 16, "D": 64, "fmt": "fp4", "masked": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "kv", "tree", "tree", "sparse", "sparse"])
    if op == "rope":
        D = rng.choice([64, 96, 128, 192, 80])
        rot = rng.choice([r for r in (16, 20, 32, 64, 96, 128, D) if r <= D])
        H = _logint(rng, 1, 64)
        scaling = rng.choice(["none", "linear", "by_parts"])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 22528 * 64 * 128 // (H * D * (2 if dtype == "fp32" else 1))
        return {"op": op, "T": _logint(rng, 1, min(22528, most)), "H": H, "D": D, "rot": rot,
                "start": rng.choice([0, D - rot]), "layout": rng.choice(["half", "interleaved"]),
                "scaling": scaling, "factor": 1.0 if scaling == "none" else float(rng.choice([2, 4, 8])),
                "dtype": dtype, "inverse": rng.random() < 0.3, "max_pos": rng.choice([32768, 131072])}
    fmt = rng.choice(["bf16", "fp8", "fp4"])
    D = rng.choice([64, 128, 128])
    if op == "kv":
        rot = rng.choice([0, 32, 64, D])
        B = _logint(rng, 1, 64)
        kv = rng.choice([1, 2, 4, 8])
        return {"op": op, "T": max(B, _logint(rng, 1, 22528)), "B": B, "kv": kv, "D": D, "fmt": fmt,
                "rot": rot, "start": rng.choice([0, D - rot]), "layout": rng.choice(["half", "interleaved"]),
                "ctx": _logint(rng, 1, 16384)}
    kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]) if rng.random() < 0.8 else rng.choice([32, 64])
    if op == "tree":
        nd = _logint(rng, 1, 96)
        ctx = _logint(rng, 1, 131072)
        # what a batch of this shape may cost: key rows read, and products
        most = min(2 ** 31 // (ctx * kv * D), 2 ** 30 // (ctx * kv * G * nd))
        return {"op": op, "B": max(1, min(_logint(rng, 1, 64), most)), "nd": nd,
                "ctx_min": max(1, ctx // rng.choice([1, 2, 8])), "ctx_max": ctx, "kv": kv, "G": G, "D": D,
                "fmt": fmt, "masked": rng.random() < 0.7}
    k = rng.choice([512, 1024, 2048, 300])
    nd = _logint(rng, 1, 64)
    most = 2 ** 30 // (nd * k * kv * max(D, G))
    ctx = _logint(rng, 64, 32768)
    return {"op": op, "B": max(1, min(_logint(rng, 1, 64), most)), "nd": nd,
            "ctx_min": max(1, ctx // rng.choice([1, 2, 8])), "ctx_max": ctx, "k": k, "kv": kv, "G": G, "D": D,
            "fmt": fmt, "masked": rng.random() < 0.5}


def _lengths(case):
    """Committed context lengths of the batch: spread evenly over the case's
    range, in an order that mixes long and short."""
    B, lo, hi = case["B"], case["ctx_min"], case["ctx_max"]
    step = next(s for s in (37, 11, 7, 5, 3, 1) if math.gcd(s, B) == 1)
    return [lo + ((b * step) % B) * (hi - lo) // max(1, B - 1) for b in range(B)]


def _row_bytes(fmt, D):
    return {"bf16": 2 * D, "fp8": D + D // BLOCK, "fp4": D // 2 + D // BLOCK}[fmt]


def work(case):
    if case["op"] == "rope":
        es = 4 if case["dtype"] == "fp32" else 2
        n = case["T"] * case["H"]
        return {"bytes": 2 * n * case["D"] * es + 4 * case["T"], "flops": 3 * n * case["rot"]}
    if case["op"] == "kv":
        rows = 2 * case["T"] * case["kv"]
        return {"bytes": rows * (2 * 2 * case["D"] + 2 * _row_bytes(case["fmt"], case["D"])) + 12 * case["T"],
                "flops": 3 * case["T"] * case["kv"] * case["rot"]}
    lens = _lengths(case)
    nd, kv, H, D = case["nd"], case["kv"], case["kv"] * case["G"], case["D"]
    row = _row_bytes(case["fmt"], D)
    io = case["B"] * nd * H * (2 * 2 * D + 4)
    if case["op"] == "tree":
        keys = sum(c + nd for c in lens)
        # each drafted token sees its context and itself; a chain also what came before it
        pairs = sum(nd * (c + 1) + (0 if case["masked"] else nd * (nd - 1) // 2) for c in lens)
    else:
        pairs = sum(nd * (min(case["k"], c) + (1 if case["masked"] else 0)) for c in lens)
        # queries of one sequence may select the same rows: a row counts once
        keys = sum(min(c, nd * min(case["k"], c)) + (nd if case["masked"] else 0) for c in lens)
        io += case["B"] * nd * case["k"] * 4
    return {"bytes": keys * kv * 2 * row + io, "flops": pairs * H * D * 4}


# ------------------------------------------------------------------ formats

def _fp4_edges(device):
    """Upper edges of the codes 0..6: a value above edge i has a code above i;
    on the edge it takes the even code."""
    e = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float32, device=device)
    below = torch.nextafter(e, torch.zeros_like(e))
    odd = torch.arange(7, device=device) % 2 == 1
    return torch.where(odd, below, e)


def _quantise(y, fmt):
    """fp32 [..., D] -> (codes uint8 [..., code bytes], scales uint8 [..., D/32] or None)."""
    if fmt == "bf16":
        return y.to(torch.bfloat16).view(torch.uint8), None
    blocks = y.reshape(*y.shape[:-1], -1, BLOCK)
    amax = blocks.abs().amax(-1)
    m, e = torch.frexp(amax)
    if fmt == "fp8":
        e = (e - 9 + (m > 0.875)).clamp(-117, 119)
    else:
        e = (e - 3 + (m > 0.75)).clamp(-125, 125)
    e = torch.where(amax == 0, torch.full_like(e, -117 if fmt == "fp8" else -125), e)
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
        pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        x = table[pair.long()]
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


def _page_bytes(case):
    """Bytes of one kv head's part of a page."""
    return 2 * PAGE * _row_bytes(case["fmt"], case["D"])


# ------------------------------------------------------------------ rotary tables

def _frequencies(rot, theta, scaling, factor, orig=32768, slow=1.0, fast=32.0):
    """Angular frequency of each pair, in double."""
    f = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / max(rot, 1))
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        keep = np.clip((orig * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep
    return f


def _magnitude(scaling, factor):
    return 0.1 * math.log(factor) + 1.0 if scaling == "by_parts" else 1.0


def _rotate(x, angle, mag, case, inverse, dtype):
    """x [T, H, D] in `dtype`, angle [T, rot/2] in double."""
    R, s = case["rot"], case["start"]
    if R == 0:
        return x
    c = (torch.cos(angle) * mag).to(dtype)[:, None, :]
    n = (torch.sin(angle) * (-mag if inverse else mag)).to(dtype)[:, None, :]
    part = x[..., s:s + R]
    if case["layout"] == "half":
        a, b = part[..., :R // 2], part[..., R // 2:]
        part = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([x[..., :s], part, x[..., s + R:]], -1)


# ------------------------------------------------------------------ the library's handles

@functools.lru_cache(maxsize=None)
def _context():
    from dsa_sparse_attention_store_gb300 import Context
    return Context(max_pos=64)


@functools.lru_cache(maxsize=None)
def _rope(rot, layout, scaling, factor, max_pos):
    from dsa_sparse_attention_store_gb300 import Rope
    return Rope(_context(), rot_dim=rot, max_pos=max_pos, theta=10000.0, layout=layout, scaling=scaling,
                factor=factor, orig_max_pos=32768, beta_slow=1.0, beta_fast=32.0,
                mscale=_magnitude(scaling, factor))


# ------------------------------------------------------------------ states

def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _paging(lens, gen):
    """A page table over randomly placed pages for sequences of these lengths."""
    pages = [-(-n // PAGE) for n in lens]
    total = sum(pages) + 3
    order = torch.randperm(total, generator=gen, device=DEV)[:sum(pages)].to(torch.int32)
    table = torch.zeros((len(lens), max(pages)), dtype=torch.int32, device=DEV)
    table[torch.arange(max(pages), device=DEV)[None, :] < _int(pages)[:, None]] = order
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


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = {"case": case}
    if case["op"] == "rope":
        T = case["T"]
        s["x"] = normal(T, case["H"], case["D"]).to(DTYPE[case["dtype"]])
        first = int(torch.randint(0, max(1, case["max_pos"] - T), (1,), generator=gen, device=DEV))
        s["pos"] = torch.arange(first, first + T, dtype=torch.int32, device=DEV)
        if own:
            s["ctx"] = _context()
            s["rope"] = _rope(case["rot"], case["layout"], case["scaling"], case["factor"], case["max_pos"])
            s["out"] = torch.empty_like(s["x"])
        return s
    kv, D = case["kv"], case["D"]
    if case["op"] == "kv":
        T, B = case["T"], case["B"]
        new = [T // B + (b < T % B) for b in range(B)]
        s["table"], s["pages"] = _paging([case["ctx"] + n for n in new], gen)
        s["seq"] = torch.repeat_interleave(torch.arange(B, device=DEV), _int(new).long()).to(torch.int32)
        s["pos"] = torch.cat([torch.arange(case["ctx"], case["ctx"] + n, device=DEV) for n in new]).to(torch.int32)
        # keys with a few large channels, as projections have them
        gain = torch.exp(normal(kv, D) * 0.7)
        s["k"] = (normal(T, kv, D) * gain).to(torch.bfloat16)
        s["v"] = normal(T, kv, D).to(torch.bfloat16)
        s["cache"] = torch.zeros((s["pages"], kv, _page_bytes(case)), dtype=torch.uint8, device=DEV)
        if own:
            s["ctx"] = _context()
            s["rope"] = _rope(case["rot"], case["layout"], "none", 1.0, 65536) if case["rot"] else None
            s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return s
    B, nd = case["B"], case["nd"]
    ctx = _lengths(case)
    s["table"], s["pages"] = _paging([c + nd for c in ctx], gen)
    s["lens"] = _int([c + nd for c in ctx])
    s["cu_q"] = _int([b * nd for b in range(B + 1)])
    s["cache"] = torch.empty((s["pages"], kv, _page_bytes(case)), dtype=torch.uint8, device=DEV)
    kc, ks, vc, vs = _fields(s["cache"], case)
    for at in range(0, s["pages"], 1024):  # a part at a time: the 32-bit values of a long context are large
        n = min(1024, s["pages"] - at)
        for codes, scales in ((kc, ks), (vc, vs)):
            c, e = _quantise(normal(n, kv, PAGE, D), case["fmt"])
            codes[at:at + n] = c
            if e is not None:
                scales[at:at + n] = e
    H = kv * case["G"]
    s["q"] = (normal(B * nd, H, D) * 2.0).to(torch.bfloat16)
    s["mask"] = _tree(B, nd, gen) if case["masked"] else None
    if case["op"] == "sparse":
        k = case["k"]
        sel = torch.full((B * nd, k), -1, dtype=torch.int32, device=DEV)
        for b, c in enumerate(ctx):  # k distinct committed positions for each query, in the order of their scores
            n = min(k, c)
            u = torch.rand((nd, c), generator=gen, device=DEV)
            sel[b * nd:(b + 1) * nd, :n] = u.topk(n, dim=1).indices.to(torch.int32)
        s["sel"] = sel
    if own:
        s["ctx"] = _context()
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B * nd, H), dtype=torch.float32, device=DEV)
        s["ws"] = torch.empty(s["ctx"].attn_workspace_size(D), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    case, ctx = s["case"], s["ctx"]
    if case["op"] == "rope":
        ctx.rope_apply(s["x"], s["pos"], s["rope"], out=s["out"], rot_start=case["start"], inverse=case["inverse"])
        return s["out"]
    cache, fmt = s["cache"].view(-1), FMT[case["fmt"]]
    if case["op"] == "kv":
        ctx.kv_store(s["k"], s["v"], s["pos"], s["seq"], s["table"], cache, s["pages"], fmt,
                     rope=s["rope"], rot_start=case["start"])
        ctx.kv_load(cache, s["pages"], fmt, s["pos"], s["seq"], s["table"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if case["op"] == "tree":
        ctx.tree_attn(s["q"], cache, s["pages"], fmt, case["kv"], s["table"], s["lens"], s["cu_q"], s["out"],
                      s["ws"], mask=s["mask"], lse=s["lse"])
    else:
        ctx.sparse_attn(s["q"], s["sel"], cache, s["pages"], fmt, case["kv"], s["table"], s["lens"], s["cu_q"],
                        s["out"], s["ws"], mask=s["mask"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rope":
        f = torch.from_numpy(_frequencies(case["rot"], 10000.0, case["scaling"], case["factor"])).to(DEV)
        y = _rotate(s["x"].float(), s["pos"].double()[:, None] * f, _magnitude(case["scaling"], case["factor"]),
                    case, case["inverse"], torch.float32)
        return y.to(s["x"].dtype)
    kc, ks, vc, vs = _fields(s["cache"], case)
    fmt = case["fmt"]
    if case["op"] == "kv":
        f = torch.from_numpy(_frequencies(case["rot"], 10000.0, "none", 1.0)).to(DEV)
        k = _rotate(s["k"].float(), s["pos"].double()[:, None] * f, 1.0, case, False, torch.float32)
        pos = s["pos"].long()
        page, off = s["table"][s["seq"].long(), pos // PAGE].long(), pos % PAGE
        at = (page[:, None], torch.arange(case["kv"], device=DEV)[None, :], off[:, None])
        back = []
        for x, codes, scales in ((k, kc, ks), (s["v"].float(), vc, vs)):
            c, e = _quantise(x, fmt)
            codes[at] = c
            if e is not None:
                scales[at] = e
            back.append(_dequantise(codes[at], None if e is None else scales[at], fmt, torch.float32).to(torch.bfloat16))
        return {"k": back[0], "v": back[1]}
    B, nd, kv, G, D = case["B"], case["nd"], case["kv"], case["G"], case["D"]
    lens = s["lens"].long()
    drafted = torch.arange(nd, device=DEV)
    if s["mask"] is not None:
        bit = (s["mask"].view(B, nd, -1, 1) >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        seen = bit.flatten(2)[..., :nd].bool()
    else:
        seen = (drafted[None, :] <= drafted[:, None]).expand(B, nd, nd)
    if case["op"] == "tree":
        # one group of keys for each sequence: [B, L]; queries of a sequence share it
        pos = torch.arange(int(case["ctx_max"] + nd), device=DEV).expand(B, -1)
        j = pos - (lens - nd)[:, None]
        see = torch.where((j < 0)[:, None, :], True,
                          seen.gather(2, j.clamp(0, nd - 1)[:, None, :].expand(-1, nd, -1))) & (j < nd)[:, None, :]
        page = s["table"].long()[torch.arange(B, device=DEV)[:, None], (pos // PAGE).clamp(max=s["table"].shape[1] - 1)]
        off = pos % PAGE
        q = s["q"].view(B, nd, kv, G, D)
    else:
        # one group of keys for each query: its selection, then the drafted tokens
        b = torch.arange(B, device=DEV).repeat_interleave(nd)
        pos, see = s["sel"].long(), s["sel"] >= 0
        if s["mask"] is not None:
            pos = torch.cat([pos, (lens - nd)[b][:, None] + drafted], 1)
            see = torch.cat([see, seen.reshape(B * nd, nd)], 1)
        pos = pos.clamp(min=0)
        page, off = s["table"].long()[b[:, None], pos // PAGE], pos % PAGE
        see = see[:, None, :]
        q = s["q"].view(B * nd, 1, kv, G, D)
    at = (page[:, None, :], torch.arange(kv, device=DEV)[None, :, None], off[:, None, :])
    n = q.shape[1]
    q = q.permute(0, 2, 1, 3, 4).reshape(q.shape[0], kv, n * G, D).float()
    see = see[:, None, :, None, :].expand(-1, 1, -1, G, -1).reshape(q.shape[0], 1, n * G, -1)
    k = _dequantise(kc[at], None if ks is None else ks[at], fmt, torch.float32)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).masked_fill_(~see, -math.inf)
    del k
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _dequantise(vc[at], None if vs is None else vs[at], fmt, torch.float32)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)
    back = lambda x: x.view(-1, kv, n, G, x.shape[-1]).transpose(1, 2).reshape(B * nd, kv * G, -1)  # noqa: E731
    return {"out": back(out).to(torch.bfloat16), "lse": back(lse).squeeze(-1)}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rope(x, pos, case, f, mag, inverse):
    """Pairs as complex numbers: (a + bi) e^(i angle)."""
    R, s = case["rot"], case["start"]
    y = x.double().clone()
    if R == 0:
        return y
    i = torch.arange(R // 2, device=DEV)
    lo, hi = (s + i, s + i + R // 2) if case["layout"] == "half" else (s + 2 * i, s + 2 * i + 1)
    turn = torch.polar(torch.full((1, R // 2), mag, dtype=torch.float64, device=DEV),
                       pos.double()[:, None] * torch.tensor(f, device=DEV) * (-1.0 if inverse else 1.0))
    z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None, :]
    y[..., lo], y[..., hi] = z.real.contiguous(), z.imag.contiguous()
    return y


def _exact_values(y, fmt):
    """What the cache stands for after y was written into it, by the formats' definition."""
    if fmt == "bf16":
        return y.to(torch.bfloat16).double()
    most, step, low = (448.0, 3, -6) if fmt == "fp8" else (6.0, 1, 0)
    z = y.unflatten(-1, (-1, BLOCK))
    e = torch.ceil(torch.log2(z.abs().amax(-1, keepdim=True).clamp(min=1e-300) / most)).clamp(-117, 119)
    x = z / torch.exp2(e)
    # spacing of the format's numbers around x: 2^(exponent - mantissa bits), no less than the smallest step
    ulp = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1e-300))).clamp(min=low) - step)
    return (torch.round(x / ulp) * ulp * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s["x"], s["pos"], case,
                           _frequencies(case["rot"], 10000.0, case["scaling"], case["factor"]),
                           _magnitude(case["scaling"], case["factor"]), case["inverse"])
    if case["op"] == "kv":
        k = _exact_rope(s["k"], s["pos"], case, _frequencies(case["rot"], 10000.0, "none", 1.0), 1.0, False)
        return {"k": _exact_values(k, case["fmt"]), "v": _exact_values(s["v"].double(), case["fmt"])}
    B, nd, kv, G, D = case["B"], case["nd"], case["kv"], case["G"], case["D"]
    out = torch.zeros((B * nd, kv * G, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B * nd, kv * G), -math.inf, dtype=torch.float64, device=DEV)
    fields = _fields(s["cache"], case)
    words = None if s["mask"] is None else s["mask"].cpu().numpy().astype(np.uint32)
    for b, c in enumerate(_lengths(case)):
        rows = slice(b * nd, (b + 1) * nd)
        where = torch.arange(c + nd, device=DEV)
        slot = s["table"][b, where // PAGE].long() * PAGE + where % PAGE
        see = torch.zeros((nd, c + nd), dtype=torch.bool, device=DEV)
        if case["op"] == "tree":
            see[:, :c] = True
        else:
            sel = s["sel"][rows].long()
            see[torch.arange(nd, device=DEV)[:, None].expand_as(sel)[sel >= 0], sel[sel >= 0]] = True
        if words is not None:
            own_bits = np.unpackbits(np.ascontiguousarray(words[rows]).view(np.uint8), axis=1, bitorder="little")[:, :nd]
            see[:, c:] = torch.from_numpy(own_bits.astype(bool)).to(DEV)
        elif case["op"] == "tree":
            see[:, c:] = torch.ones((nd, nd), device=DEV).tril().bool()
        for h in range(kv):
            flat = [None if x is None else x[:, h].flatten(0, 1)[slot] for x in fields]
            k, v = (_dequantise(flat[i], flat[i + 1], case["fmt"], torch.float64) for i in (0, 2))
            heads = slice(h * G, (h + 1) * G)
            q = s["q"][rows, heads].double().reshape(nd * G, D)
            z = (q @ k.T / math.sqrt(D)).masked_fill(~see.repeat_interleave(G, 0), -math.inf)
            total = torch.logsumexp(z, -1)
            w = torch.exp(z - torch.where(torch.isfinite(total), total, torch.zeros_like(total))[:, None])
            out[rows, heads] = (w @ v).view(nd, G, D)
            lse[rows, heads] = total.view(nd, G)
    return {"out": out, "lse": lse}
