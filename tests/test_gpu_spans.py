"""Attention of spans and behind shared prefixes on the GPU against the 64-bit
reference: caps, distance bias, documents, prefixes, windows, tree bits, rows
that see nothing, hidden values, bad pages and groups, streams, graphs, buffers
with canaries."""
import numpy as np
import pytest

from oracle import attention as A
from tests.span_util import SpanCase

pytestmark = pytest.mark.gpu

FMTS = [A.BF16, A.FP8, A.FP4]


@pytest.fixture(scope="module")
def ctx():
    import torch
    from dsa_sparse_attention_store_gb300 import Context
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    c = Context(max_pos=64)
    yield c
    c.close()


# few rows, up to 128 rows, and the wide form
SIZES = {
    "first": ([0], [1], 1, 1),
    "few": ([338, 64, 0], [5, 1, 3], 1, 4),
    "tree": ([700, 130, 63], [20, 9, 1], 2, 7),
    "wide": ([500, 0, 70], [60, 33, 40], 1, 8),
}


def _documents(c, part):
    """First places that cut each sequence into documents of `part` tokens and, every third, one."""
    place = c.place()
    return np.where(place % 3 == 0, place, place - place % part)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("mods", ["none", "cap", "low cap", "bias", "cap and bias", "window", "documents", "prefix", "tree"])
def test_span_matches_reference(ctx, fmt, D, size, mods):
    c = SpanCase(sum(map(ord, size + mods)), *SIZES[size], D, fmt, masked=mods == "tree",
                 cap={"cap": 30.0, "low cap": 1.5, "cap and bias": 20.0, "tree": 50.0}.get(mods, 0.0),
                 slopes="bias" in mods or None, window={"window": 70, "tree": 65}.get(mods, 0))
    if mods == "documents":
        c.mods["first"] = _documents(c, 100).astype(np.int32)
    if mods == "prefix":
        n = np.repeat(np.array(c.ctx) + np.array(c.nds) // 2, c.nds)
        c.mods["last"] = np.maximum(c.place() + 1, n).astype(np.int32)
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("nds", [[3, 9], [120, 37]])
@pytest.mark.parametrize("seed", range(4))
def test_any_spans(ctx, fmt, nds, seed):
    # spans that have nothing to do with each other or with where the token is: behind it,
    # ahead of it, empty, one key, past the end, negative
    rng = np.random.default_rng(seed)
    c = SpanCase(seed, [400, 5], nds, 2, 3, 64, fmt, cap=[0.0, 20.0][seed % 2], slopes=[None, True][seed // 2])
    L = np.repeat(c.lens, nds)
    first = rng.integers(-3, L + 3)
    last = first + rng.integers(-2, 200, len(L)) * rng.integers(0, 2, len(L))
    last[::4] = first[::4] + 1
    c.mods.update(first=first.astype(np.int32), last=last.astype(np.int32))
    out, lse = c.run(ctx)
    c.check(out, lse)
    empty = ~np.isfinite(c.reference()[1])
    assert empty.any() and np.all(out.float().cpu().numpy()[empty] == 0)
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_extremes_of_caps_and_slopes(ctx, fmt):
    # scores far beyond the cap, all at it; slopes that leave only the nearest keys, negative ones
    for kw in (dict(cap=0.01, q_gain=100.0), dict(cap=1e6), dict(cap=8.0, q_gain=0.0), dict(slopes=np.full(4, 40.0)),
               dict(slopes=np.array([-0.02, 0.0, 1e-3, 5.0]), cap=10.0)):
        c = SpanCase(17, [900], [6], 1, 4, 128, fmt, **kw)
        c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", ["few", "tree", "wide"])
@pytest.mark.parametrize("cap", [8.0, 45.0, 57.0, 62.0, 63.0, 90.0, 2000.0, 1e5])
def test_every_treatment_of_caps(ctx, fmt, size, cap):
    # weighed under one exponent (to 62), under a running maximum; scores for the polynomial, and beyond it
    for q_gain in (1.0, 12.0):
        c = SpanCase(int(cap) + int(q_gain), *SIZES[size], 64, fmt, cap=cap, q_gain=q_gain)
        c.check(*c.run(ctx))
    assert ctx.device_status() == 0


def test_far_keys_alone(ctx):
    # a bias of thousands that every visible key has: weights depend on their differences
    c = SpanCase(18, [20000], [4], 1, 2, 64, A.BF16, slopes=np.array([0.5, 0.07]), first=[100, 0, 300, 64], last=[230, 64, 310, 65])
    c.check(*c.run(ctx))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", [1, 16])
def test_windows_over_many_pages(ctx, fmt, G):
    # units whose first tile is not the sequence's, divided among many CTAs
    c = SpanCase(19, [9000, 300], [70, 2], 1, G, 128, fmt, window=5000, cap=50.0)
    c.check(*c.run(ctx))


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences(ctx, fmt):
    rng = np.random.default_rng(5)
    c = SpanCase(20, rng.integers(0, 90, 700).tolist(), rng.integers(0, 3, 700).tolist(), 1, 2, 64, fmt, cap=20.0, window=50)
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


GROUPS = [
    ([200, 300, 129], [1, 1, 1], 1, 4, [(3, 128)]),
    ([200, 300, 129], [1, 1, 1], 1, 4, [(3, 127)]),                    # shared in part: one page of two
    ([64, 64], [1, 2], 2, 1, [(2, 64)]),                               # nothing of their own before the new tokens
    ([500, 700, 40, 300, 256, 256], [3, 1, 2, 4, 1, 9], 2, 3, [(2, 450), (1, 0), (3, 256)]),
    ([130, 140, 150], [0, 3, 0], 1, 8, [(3, 128)]),                    # members without new tokens
    ([1000] * 9 + [100], [4] * 9 + [1], 2, 4, [(9, 960), (1, 64)]),    # 144 rows a group: the wide form, the sequences in the few-row one
    ([700] * 5, [40] * 5, 1, 8, [(5, 640)]),                           # wide both ways
    ([2100] * 33, [1] * 33, 1, 2, [(33, 2048)]),
    ([300, 310, 30, 20], [2, 2, 1, 1], 1, 4, [(2, 256), (0, 999), (2, 10)]),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", range(len(GROUPS)))
@pytest.mark.parametrize("mods", ["none", "cap", "bias and window", "tree"])
def test_shared_matches_reference(ctx, fmt, D, which, mods):
    ctx_lens, nds, kv, G, groups = GROUPS[which]
    c = SpanCase(100 + which, ctx_lens, nds, kv, G, D, fmt, groups=groups, masked=mods == "tree", cap=25.0 if mods in ("cap", "tree") else 0.0,
                 slopes=True if mods == "bias and window" else None, window=90 if mods == "bias and window" else 0)
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_spans_across_the_prefix(ctx, fmt):
    # documents that end inside it, rows that see only it, only what follows, or nothing
    rng = np.random.default_rng(8)
    c = SpanCase(31, [600, 520, 900], [7, 30, 4], 1, 4, 128, fmt, groups=[(3, 512)], cap=30.0, slopes=True)
    L = np.repeat(c.lens, c.nds)
    first = rng.integers(0, L)
    last = np.minimum(first + rng.integers(0, 300, len(L)), L)
    c.mods.update(first=first.astype(np.int32), last=last.astype(np.int32))
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_drafted_tokens_inside_the_prefix(ctx, fmt):
    # a shared length that passes a member's committed context, and one that passes the first sequence:
    # rows still see what their lengths and bits say
    c = SpanCase(32, [100, 300, 40], [60, 2, 90], 1, 3, 64, fmt, groups=[(3, 128)], masked=True)
    c.check(*c.run(ctx))
    c = SpanCase(32, [130, 300, 200], [2, 2, 1], 1, 3, 64, fmt, groups=[(3, 128)])
    c.shared[0] = 1 << 30                       # counts as the first sequence's 132
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_a_prefix_that_is_all_there_is(ctx, fmt, cap):
    # nothing behind the shared pages, which fill the rows of the page table: the own pass has no keys
    for seed, ctx_lens, nds, kv, D, window in ((34, [127, 125, 126], [1, 3, 2], 2, 64, 0), (35, [191, 191], [1, 1], 1, 128, 70)):
        whole = ctx_lens[0] + nds[0]
        c = SpanCase(seed, ctx_lens, nds, kv, 4, D, fmt, groups=[(len(nds), whole)], cap=cap, window=window)
        c.table = np.ascontiguousarray(c.table[:, :whole // 64])
        c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_bad_groups_are_reported_and_share_nothing(ctx, fmt):
    c = SpanCase(33, [200, 300, 129, 64], [1, 1, 1, 2], 1, 4, 64, fmt, groups=[(2, 128), (2, 64)])
    ref = c.reference()
    d = c.device()
    for cu, shared, status in (([0, 2, 9], [128, 64], 4), ([0, 3, 2], [128, 64], 4), ([-1, 2, 4], [128, 64], 4), ([0, 2, 4], [128, -5], 4),
                               ([0, 2, 2], [128, 64], 0), ([1, 2, 4], [128, 64], 0)):
        import torch
        d["cu_groups"], d["shared"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, shared))
        out, lse = c.run(ctx, d=d)
        assert ctx.device_status() == status, cu
        if cu != [0, 3, 2]:                     # a group that overlaps another's sequences may share what they do not have
            c.check(out, lse, ref=ref)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("groups", [None, [(2, 64)]])
def test_hidden_values_do_not_reach_a_row(ctx, fmt, groups):
    # keys and values that are not finite, before a window, after a span, in stale places
    c = SpanCase(41, [200, 150], [4, 40], 2, 4, 64, fmt, groups=groups, cap=20.0)
    place = c.place()
    c.mods["first"] = np.where(np.arange(c.Tq) % 5 == 0, 0, 40).astype(np.int32)
    c.mods["last"] = np.where(np.arange(c.Tq) % 7 == 3, 100, place + 1).astype(np.int32)
    clean = c.reference()
    kc, ks, vc, vs = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)
    hidden = np.ones((c.pages, 64), bool)
    for b in range(c.B):
        pos = np.arange(c.lens[b])
        hidden[c.table[b, pos // 64], pos % 64] = False
    for b in range(c.B):                        # and a place that some tokens see, of each sequence
        for pos in (7, 120):
            hidden[c.table[b, pos // 64], pos % 64] = True
    for codes, scales in ((kc, ks), (vc, vs)):
        if fmt == A.BF16:
            codes.view(np.uint16).transpose(0, 2, 1, 3)[hidden] = 0x7F80
        else:
            scales.transpose(0, 2, 1, 3)[hidden] = 255
    out, lse = c.run(ctx)
    rows = np.nonzero((c.mods["first"] == 40) & (c.mods["last"] == 100))[0]
    assert len(rows) > 2
    c.check(out, lse, ref=clean, rows=rows)
    got, want = out.double().cpu().numpy(), c.reference()[0]
    assert np.array_equal(np.isfinite(got), np.isfinite(want)) and not np.isfinite(want).all()
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("groups", [None, [(2, 256)]])
def test_bad_pages_and_lengths_are_reported_and_left_out(ctx, fmt, groups):
    c = SpanCase(61, [1000, 300, 90], [2, 1, 3], 2, 4, 64, fmt, groups=groups, cap=20.0)
    c.mods["last"] = np.minimum(c.place() + 1, 192).astype(np.int32)     # what is asked of the bad page: nothing
    ref = c.reference()
    c.mods["last"] = np.minimum(c.place() + 1, 256).astype(np.int32)
    c.table[0, 3] = c.pages + 9
    if groups:
        c.table[1, 3] = c.pages + 9
    out, lse = c.run(ctx)
    assert ctx.device_status() == 4 and ctx.device_status() == 0
    c.check(out, lse, ref=ref, rows=[0, 1, 3, 4, 5])
    # a sequence with fewer keys than queries: its rows stay as they were, the others are right
    c = SpanCase(62, [100, 300, 200], [2, 1, 1], 2, 4, 64, fmt, groups=None if groups is None else [(3, 64)])
    ref = c.reference()
    c.lens[1] = 0
    out, lse = c.run(ctx)
    assert ctx.device_status() == 4
    c.check(out, lse, ref=ref, rows=[0, 1, 3])
    assert (out[2] == 77.0).all() and (lse[2] == 77.0).all()


@pytest.mark.parametrize("groups", [None, [(3, 128)]])
def test_strides(ctx, groups):
    import torch
    c = SpanCase(71, [300, 140, 200], [5, 1, 2], 2, 4, 128, A.BF16, groups=groups, cap=30.0)
    d = c.device()
    packed = torch.randn((c.Tq, 2 * c.H, c.D), device="cuda").bfloat16()
    packed[:, c.H:] = d["q"]
    for q in (packed[:, c.H:], d["q"].transpose(0, 1).contiguous().transpose(0, 1)):
        for out in (torch.full((c.H, c.Tq, c.D), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1),
                    torch.full((c.Tq, c.H, c.D + 8), 3.0, dtype=torch.bfloat16, device="cuda")[:, :, :c.D]):
            c.check(*c.run(ctx, out=out, q=q, d=d))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("groups", [None, [(2, 768), (1, 0)]])
def test_no_writes_outside_buffers(ctx, fmt, groups):
    import torch
    c = SpanCase(81, [900, 800, 2000], [3, 1, 30], 2, 5, 128, fmt, groups=groups, window=1000)
    pad = 4096

    def padded(n):
        whole = torch.full((n + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
        return whole, whole[pad:pad + n]

    ow, o = padded(c.Tq * c.H * c.D * 2)
    lw, le = padded(c.Tq * c.H * 4)
    ww, ws = padded(c.workspace_size(ctx))
    d = c.device()
    keep = d["cache"].clone()
    c.check(*c.run(ctx, out=o.view(torch.bfloat16).view(c.Tq, c.H, c.D), lse=le.view(torch.float32).view(c.Tq, c.H), ws=ws, d=d))
    for w in (ow, lw, ww):
        assert torch.all(w[:pad] == 0x5A) and torch.all(w[-pad:] == 0x5A)
    assert torch.equal(d["cache"], keep)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("groups", [None, [(3, 512)]])
def test_repeats_streams_and_graphs_give_the_same_bits(ctx, fmt, groups):
    import torch
    c = SpanCase(91, [3000, 700, 600], [4, 9, 1], 2, 8, 128, fmt, groups=groups, cap=50.0, window=2000)
    d = c.device()
    out, lse = c.run(ctx, d=d)
    c.check(out, lse)
    ws = torch.empty(c.workspace_size(ctx), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    with torch.cuda.stream(s):
        for _ in range(3):
            c.run(ctx, out=o2, lse=l2, ws=ws, d=d)
    s.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o2.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.run(ctx, out=o2, lse=l2, ws=ws, d=d)
    # other queries, lengths and spans in the same buffers
    d["q"].copy_(d["q"].roll(1, 0))
    c.q = np.roll(c.q, 1, 0)
    d["lens"].sub_(40)
    c.lens = c.lens - 40
    c.ctx = [x - 40 for x in c.ctx]
    g.replay()
    torch.cuda.synchronize()
    c.check(o2, l2)
    assert ctx.device_status() == 0


def test_no_prefix_is_span_attn_and_no_span_is_tree_attn(ctx):
    # the same kernels and sums where nothing is shared; tree_attn's within the same tolerance
    import torch
    c = SpanCase(95, [700, 60], [2, 5], 1, 4, 64, A.FP8, groups=[(1, 640), (1, 0)])
    d = c.device()
    out, lse = c.run(ctx, d=d)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(c.workspace_size(ctx), dtype=torch.uint8, device="cuda")
    args = (d["q"], d["cache"], c.pages, c.fmt, 1, d["table"], d["lens"], d["cu"])
    ctx.span_attn(*args, o2, ws, lse=l2, scale=c.scale)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    ctx.span_attn(*args, o2, ws, scale=c.scale)                          # without lse
    assert torch.equal(out, o2)
    ctx.tree_attn(*args, o2, ws, lse=l2, scale=c.scale)
    c.check(o2, l2)
    ctx.span_attn(d["q"][:0], *args[1:5], d["table"][:1], d["lens"][1:], d["cu"][:2] * 0, o2[:0], ws)
    ctx.shared_attn(d["q"][:0], *args[1:5], d["table"][:1], d["lens"][1:], d["cu"][:2] * 0, o2[:0], ws, d["cu_groups"][:2], d["shared"][:1])
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("groups", [None, [(2, 192)]])
def test_padded_batches_leave_the_rows_behind_as_they_were(ctx, fmt, groups):
    # more rows of q than the sequences have
    import torch
    c = SpanCase(93, [300, 200], [3, 40], 2, 4, 64, fmt, groups=groups, cap=30.0, window=120)
    d = c.device()
    pad = 37
    d["q"] = torch.cat([d["q"], torch.full((pad, c.H, c.D), float("nan"), dtype=torch.bfloat16, device="cuda")])
    rows, c.Tq = c.Tq, c.Tq + pad
    out, lse = c.run(ctx, d=d)
    c.Tq = rows
    c.check(out[:rows], lse[:rows])
    assert (out[rows:] == 77.0).all() and (lse[rows:] == 77.0).all()
    assert ctx.device_status() == 0


@pytest.mark.parametrize("groups", [None, [(4, 640)]])
def test_calls_on_two_streams_at_once(ctx, groups):
    # each with a workspace of its own
    import torch
    cs = [SpanCase(94 + i, [700 + 100 * i, 900, 650, 800], [5, 1, 30, 2], 2, 8, 128, A.FP8, groups=groups, cap=[0.0, 40.0][i]) for i in range(2)]
    ds = [c.device() for c in cs]
    wants = [c.run(ctx, d=d) for c, d in zip(cs, ds)]
    outs = [[torch.empty_like(x) for x in w] for w in wants]
    wss = [torch.empty(c.workspace_size(ctx), dtype=torch.uint8, device="cuda") for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, d, o, ws, s in zip(cs, ds, outs, wss, streams):
            with torch.cuda.stream(s):
                c.run(ctx, out=o[0], lse=o[1], ws=ws, d=d)
    torch.cuda.synchronize()
    for c, w, o in zip(cs, wants, outs):
        c.check(*w)
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_cache_past_32_bits(ctx, fmt):
    # a cache of more than 4 GB, the sequences' pages at its far end
    import torch
    from dsa_sparse_attention_store_gb300 import kv_page_bytes
    c = SpanCase(99, [300, 200], [2, 1], 4, 2, 128, fmt, groups=[(2, 192)], cap=30.0)
    pb = kv_page_bytes(4, 128, fmt)
    shift = (1 << 32) // pb + 10
    d = c.device()
    big = torch.empty((shift + c.pages) * pb, dtype=torch.uint8, device="cuda")
    big[shift * pb:] = d["cache"]
    d["cache"] = big
    d["table"] = torch.where(d["table"] < (1 << 29), d["table"] + shift, d["table"])
    small, c.pages = c.pages, shift + c.pages
    out, lse = c.run(ctx, d=d)
    c.pages = small
    c.check(out, lse)
    assert ctx.device_status() == 0


def test_binding_refusals(ctx):
    import torch
    from dsa_sparse_attention_store_gb300 import dsaidx
    c = SpanCase(97, [150, 150], [2, 1], 1, 4, 64, A.BF16, groups=[(2, 128)], slopes=True)
    d = c.device()
    out, lse = c.run(ctx, d=d)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(c.workspace_size(ctx), dtype=torch.uint8, device="cuda")

    def shared(**kw):
        a = dict(q=d["q"], cache=d["cache"], num_pages=c.pages, fmt=c.fmt, kv_heads=1, page_table=d["table"], seq_lens=d["lens"],
                 cu_q=d["cu"], out=out, workspace=ws, cu_groups=d["cu_groups"], shared_lens=d["shared"], lse=lse)
        a.update(kw)
        ctx.shared_attn(**a)

    shared()
    for kw, err in [(dict(first=i32(2)), ValueError), (dict(last=i32(3).long()), TypeError), (dict(slopes=d["slopes"][:2]), ValueError),
                    (dict(slopes=d["slopes"].double()), TypeError), (dict(cu_groups=i32(3)), ValueError),
                    (dict(shared_lens=d["shared"].cpu()), TypeError), (dict(first=i32(6)[::2]), ValueError)]:
        with pytest.raises(err):
            shared(**kw)
    for kw, status in [(dict(workspace=ws[:-1]), 6), (dict(cap=-1.0), 1), (dict(cap=float("nan")), 1), (dict(window=-1), 1),
                       (dict(slopes=d["slopes"], mask=i32(3, 1)), 2)]:
        with pytest.raises(dsaidx.DsaError) as e:
            shared(**kw)
        assert e.value.status == status, kw
    with pytest.raises(dsaidx.DsaError) as e:
        ctx.span_attn(d["q"], d["cache"], c.pages, c.fmt, 1, d["table"], d["lens"], d["cu"], out,
                      ws[:ctx.span_attn_workspace_size(3, 2, 4, 1, 64) - 1])
    assert e.value.status == 6
    shared()
    assert ctx.device_status() == 0
