"""Attention over the K/V cache on the GPU against the 64-bit reference: tree
and selection forms in every cache format, ragged and empty, masks that leave
a row nothing, values that are not finite where a row must not see them, bad
pages, streams, graphs, canaries around every buffer."""
import numpy as np
import pytest

from oracle import attention as A

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


class Case:
    """A batch: lens committed tokens and nd new ones per sequence, a random
    cache, queries, optional tree masks and selections."""

    def __init__(self, seed, ctx_lens, nds, kv, G, D, fmt, masked=True, k=None, q_gain=1.0):
        rng = np.random.default_rng(seed)
        self.kv, self.G, self.D, self.fmt, self.H = kv, G, D, fmt, kv * G
        self.nds, self.ctx = list(nds), list(ctx_lens)
        self.lens = np.array([c + n for c, n in zip(ctx_lens, nds)], np.int32)
        self.cu = np.concatenate([[0], np.cumsum(nds)]).astype(np.int32)
        self.Tq, self.B = int(self.cu[-1]), len(nds)
        pages = [max(1, -(-int(n) // 64)) for n in self.lens]
        self.pages = sum(pages) + 3
        order = rng.permutation(self.pages)
        self.table = np.full((self.B, max(pages) + 1), 1 << 30, np.int32)   # entries past a sequence's end are not read
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = A.random_cache(rng, self.pages, kv, D, fmt)
        q = (rng.standard_normal((self.Tq, self.H, D)) * q_gain).astype(np.float32)
        self.q = A.bf16_value(A.bf16_bits(q))
        self.mask = None
        if masked:
            nmax = max(nds)
            words = -(-nmax // 32)
            bits = np.zeros((self.Tq, words * 32), bool)
            for b in range(self.B):
                n, r0 = nds[b], self.cu[b]
                for i in range(n):
                    if i:
                        bits[r0 + i] = bits[r0 + rng.integers(max(0, i - 3), i)]
                    bits[r0 + i, i] = True
            self.bits = bits
            self.mask = self._pack(bits)
        self.sel = None
        if k:
            self.sel = np.full((self.Tq, k), -1, np.int32)
            for b in range(self.B):
                for t in range(self.cu[b], self.cu[b + 1]):
                    n = min(k, self.ctx[b])
                    self.sel[t, :n] = rng.permutation(self.ctx[b])[:n]
        self.scale = D ** -0.5

    @staticmethod
    def _pack(bits):
        return np.ascontiguousarray(np.packbits(bits, axis=1, bitorder="little")).view(np.uint32).copy()

    def set_bits(self, bits):
        self.bits, self.mask = bits, self._pack(bits)

    def device(self):
        import torch
        d = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.d = dict(q=d(self.q).bfloat16(), cache=d(self.cache), table=d(self.table), lens=d(self.lens), cu=d(self.cu),
                      mask=None if self.mask is None else d(self.mask.view(np.int32)), sel=d(self.sel))
        return self.d

    def run(self, ctx, out=None, lse=None, ws=None, q=None, stream=None, d=None):
        import torch
        d = self.device() if d is None else d
        q = d["q"] if q is None else q
        out = torch.full((self.Tq, self.H, self.D), 77.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        lse = torch.full((self.Tq, self.H), 77.0, device="cuda") if lse is None else lse
        if ws is None:
            # a workspace's old contents are scratch: NaN patterns must not matter
            ws = torch.full((ctx.attn_workspace_size(self.D),), 0xFF, dtype=torch.uint8, device="cuda")
        args = (d["cache"], self.pages, self.fmt, self.kv, d["table"], d["lens"], d["cu"], out, ws)
        if self.sel is None:
            ctx.tree_attn(q, *args, mask=d["mask"], lse=lse, scale=self.scale, stream=stream)
        else:
            ctx.sparse_attn(q, d["sel"], *args, mask=d["mask"], lse=lse, scale=self.scale, stream=stream)
        return out, lse

    def reference(self, slots=False, sel=None):
        keys, vals = A.values(self.cache, self.pages, self.kv, self.D, self.fmt)
        return A.attend(self.q.astype(np.float64), self.kv, keys, vals, self.table, self.lens, self.cu, self.scale, self.mask,
                        self.sel if sel is None else sel, slots)

    def check(self, out, lse, ref=None, rows=None):
        o, z, wabs, qk = self.reference() if ref is None else ref
        to, tl = A.tolerance(o, z, wabs, qk, self.scale, self.D, float(self.lens.max()))
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        rows = slice(None) if rows is None else rows
        fin = np.isfinite(z[rows])
        assert np.array_equal(gl[rows][~fin], z[rows][~fin])
        assert np.all(np.abs(gl[rows][fin] - z[rows][fin]) <= tl[rows][fin]), float(np.max((np.abs(gl[rows] - z[rows]) / tl[rows])[fin]))
        err = np.abs(got[rows] - o[rows])
        assert np.all(err <= to[rows]), (float(np.max(err / to[rows])), np.argwhere(~(err <= to[rows]))[:5].tolist())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx_lens,nds,kv,G", [
    ([0], [1], 1, 1),                          # the first token of all
    ([5], [1], 1, 1),
    ([64], [1], 2, 3),                         # a page boundary under the new token
    ([63], [1], 1, 8),
    ([338], [5], 1, 16),
    ([200, 0, 1000, 63, 64], [1, 3, 2, 1, 9], 2, 4),
    ([700, 130], [40, 33], 1, 7),              # rows past one tile, G not a power of two
    ([129], [128], 2, 1),
    ([4509], [1], 8, 8),
])
def test_tree_matches_reference(ctx, fmt, D, ctx_lens, nds, kv, G):
    c = Case(hash((fmt, D, kv, G, len(nds))) % 10000, ctx_lens, nds, kv, G, D, fmt)
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_chain_matches_reference(ctx, fmt, D):
    # no mask: a chunk of a prefill; query tiles end inside tokens (G = 3)
    c = Case(7, [0, 1000, 77], [150, 100, 1], 2, 3, D, fmt, masked=False)
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx_lens,nds,kv,G,masked", [
    ([0, 500, 0], [33, 70, 1], 1, 8, True),     # units of 264, 560 and 8 rows: whole, part of and none of the second group
    ([1000], [17], 2, 16, True),                # 272 rows: the last unit has 16
    ([2000, 300], [100, 64], 1, 12, False),
    ([64, 128], [96, 160], 4, 2, False),        # rows that end with the tiles
    ([5000], [130], 1, 3, True),                # a unit divided among many CTAs
])
def test_wide_units_match_reference(ctx, fmt, D, ctx_lens, nds, kv, G, masked):
    c = Case(hash((fmt, D, kv, G, len(nds), 2)) % 10000, ctx_lens, nds, kv, G, D, fmt, masked=masked)
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("q_gain", [0.0, 8.0])
def test_flat_and_peaked_scores(ctx, fmt, q_gain):
    # all weights equal, and weights that one key dominates (the running maximum moves late)
    c = Case(11, [3000], [2], 1, 4, 128, fmt, q_gain=q_gain)
    c.check(*c.run(ctx))


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences_and_many_pieces(ctx, fmt):
    # more sequences than threads of a block plan in one step; and one long
    # sequence divided among every CTA (more than the few pieces a warp joins)
    rng = np.random.default_rng(1)
    c = Case(12, rng.integers(0, 90, 700).tolist(), rng.integers(0, 3, 700).tolist(), 1, 2, 64, fmt)
    c.check(*c.run(ctx))
    c = Case(13, [22528], [3], 1, 5, 128, fmt)
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx_lens,nds,kv,G,k,masked", [
    ([300], [1], 1, 64, 512, False),           # fewer keys than the selection
    ([2000], [3], 2, 8, 512, True),
    ([1000, 0, 70, 5000], [1, 2, 1, 5], 1, 16, 300, True),
    ([500, 900], [30, 41], 4, 1, 64, False),
    ([700], [2], 1, 128, 1, False),
    ([4000], [33], 2, 3, 130, True),
])
def test_selection_matches_reference(ctx, fmt, D, ctx_lens, nds, kv, G, k, masked):
    c = Case(hash((fmt, D, kv, G, k)) % 10000, ctx_lens, nds, kv, G, D, fmt, masked=masked, k=k)
    c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_selection_by_slots_and_with_repeats(ctx, fmt):
    c = Case(21, [900, 300], [3, 2], 2, 4, 128, fmt, masked=False, k=200)
    c.sel[1, 5:9] = c.sel[1, 4]                 # a key listed five times counts five times
    c.sel[0, ::3] = -1                          # gaps
    c.sel[4] = -1                               # nothing selected
    c.check(*c.run(ctx))
    pos = c.sel
    b = np.searchsorted(c.cu, np.arange(c.Tq), side="right") - 1
    c.sel = np.where(pos >= 0, c.table[b[:, None], np.maximum(pos, 0) // 64] * 64 + pos % 64, -1).astype(np.int32)
    ctx.set_slot_output(True)
    try:
        out, lse = c.run(ctx)
        c.check(out, lse, ref=c.reference(slots=True))
        assert ctx.device_status() == 0
        c.sel[2, 0] = c.pages * 64              # a slot past the cache: left out, reported
        want = c.sel.copy()
        want[2, 0] = -1
        out, lse = c.run(ctx)
        assert ctx.device_status() == 4
        c.check(out, lse, ref=c.reference(slots=True, sel=want))
    finally:
        ctx.set_slot_output(False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ctx_len", [0, 40, 130])
def test_rows_that_see_nothing(ctx, fmt, ctx_len):
    c = Case(31, [ctx_len, 70], [6, 2], 2, 4, 64, fmt)
    bits = c.bits.copy()
    bits[2] = False                             # nothing of the tree
    bits[4] = False
    bits[4, 40 % bits.shape[1]] = True          # a bit past the drafted tokens: nothing
    c.set_bits(bits)
    out, lse = c.run(ctx)
    c.check(out, lse)
    if ctx_len == 0:
        import torch
        assert torch.all(out[2] == 0) and torch.all(lse[2] == -float("inf")) and torch.all(out[4] == 0)
    assert ctx.device_status() == 0


def _poison(c, b, j, what, part="v", dims=slice(0, 40)):
    """Drafted token j of sequence b holds values that are not finite."""
    kc, ks, vc, vs = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)
    pos = c.ctx[b] + j
    p, o = c.table[b, pos // 64], pos % 64
    codes, scales = (kc, ks) if part == "k" else (vc, vs)
    if c.fmt == A.BF16:
        codes.view(np.uint16)[p, :, o, dims] = {"nan": 0x7FC1, "inf": 0x7F80, "-inf": 0xFF80, "low": 0xFF7F}[what]
    else:
        scales[p, :, o, 0] = 255


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what,part", [("nan", "v"), ("inf", "v"), ("-inf", "v"), ("nan", "k"), ("inf", "k"), ("low", "k"), ("low", "v")])
def test_hidden_values_do_not_reach_a_row(ctx, fmt, D, what, part):
    if fmt != A.BF16 and what != "nan":
        pytest.skip("fp8 and fp4 blocks hold NaN or finite values")
    c = Case(41, [100, 30], [7, 3], 2, 4, D, fmt)
    bits = c.bits.copy()
    bits[:7, 3] = False
    bits[3, 3] = True                           # only token 3 of sequence 0 sees itself
    c.set_bits(bits)
    clean = c.reference()
    _poison(c, 0, 3, what, part)
    out, lse = c.run(ctx)
    rows = [0, 1, 2, 4, 5, 6, 7, 8, 9]
    c.check(out, lse, ref=clean, rows=rows)
    if part == "v":                             # and the row that sees it shows it, in those dimensions only
        o, z, wabs, qk = c.reference()
        got = out[3].double().cpu().numpy()
        if what == "low":
            assert np.all(np.sign(got[:, :32]) == np.sign(o[3][:, :32]))
            return
        n = 32 if fmt != A.BF16 else 40
        assert np.array_equal(np.isnan(got), np.isnan(o[3])) and np.array_equal(np.isposinf(got), np.isposinf(o[3]))
        assert not np.any(np.isfinite(got[:, :n])) and np.all(np.isfinite(got[:, n:]))
        assert np.all(np.abs(got[:, n:] - clean[0][3][:, n:]) <= A.tolerance(*clean, c.scale, D, 200.0)[0][3][:, n:])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx_len", [0, 100, 130, 199])
def test_hidden_values_in_wide_units(ctx, fmt, D, ctx_len):
    # 70 drafted tokens, 280 rows; a committed token and a drafted one hold
    # what is not finite in the same 128-key tile as keys others do not see
    c = Case(43, [ctx_len], [70], 1, 4, D, fmt)
    bits = c.bits.copy()
    bits[:, 9] = False
    bits[9, 9] = bits[60, 9] = True
    c.set_bits(bits)
    clean = c.reference()
    _poison(c, 0, 9, "nan")
    out, lse = c.run(ctx)
    rows = [i for i in range(70) if i not in (9, 60)]
    c.check(out, lse, ref=clean, rows=rows)
    got, o = out.double().cpu().numpy(), c.reference()[0]
    assert np.array_equal(np.isnan(got), np.isnan(o)) and np.isnan(got[9]).any() and np.isnan(got[60]).any()
    if ctx_len:                                 # a committed token is seen by every row
        _poison(c, 0, -3, "nan")
        out, lse = c.run(ctx)
        got, o = out.double().cpu().numpy(), c.reference()[0]
        assert np.array_equal(np.isnan(got), np.isnan(o)) and np.isnan(got).any(-1).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("sparse", [False, True])
def test_stale_places_do_not_matter(ctx, fmt, sparse):
    # every place past a sequence's end holds NaN, the rest of its last page and whole unused pages
    c = Case(51, [100, 64, 10], [2, 1, 1], 1, 8, 128, fmt, k=100 if sparse else None)
    ref = c.reference()
    used = np.zeros((c.pages, 64), bool)
    for b in range(c.B):
        pos = np.arange(c.lens[b])
        used[c.table[b, pos // 64], pos % 64] = True
    kc, ks, vc, vs = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)
    for codes, scales in ((kc, ks), (vc, vs)):
        if fmt == A.BF16:
            codes.view(np.uint16).transpose(0, 2, 1, 3)[~used] = 0x7FC0
        else:
            scales.transpose(0, 2, 1, 3)[~used] = 255
    out, lse = c.run(ctx)
    c.check(out, lse, ref=ref)


@pytest.mark.parametrize("fmt", FMTS)
def test_query_that_is_not_finite_stays_in_its_row(ctx, fmt):
    import torch
    c = Case(55, [500], [4], 1, 8, 128, fmt)
    ref = c.reference()
    d = c.device()
    d["q"][1, 3] = float("nan")
    d["q"][2, 0, 5] = float("inf")
    out, lse = c.run(ctx, d=d)
    got, gl = out.clone(), lse.clone()
    assert torch.all(got[1, 3].isnan()) and torch.all(got[2, 0].isnan())
    want = torch.from_numpy(ref[0]).cuda()
    got[1, 3], got[2, 0] = want[1, 3].bfloat16(), want[2, 0].bfloat16()
    gl[1, 3], gl[2, 0] = float(ref[1][1, 3]), float(ref[1][2, 0])
    c.check(got, gl, ref=ref)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("sparse", [False, True])
def test_bad_pages_and_lengths_are_reported_and_left_out(ctx, fmt, sparse):
    c = Case(61, [1000, 300], [2, 1], 2, 4, 64, fmt, k=400 if sparse else None)
    full = c.table.copy()
    c.table[0, 3] = c.pages + 9                 # positions 192..255 of sequence 0
    c.table[0, 7] = -4
    out, lse = c.run(ctx)
    assert ctx.device_status() == 4 and ctx.device_status() == 0
    # the reference leaves those keys out: as a selection without them
    bad = set(range(192, 256)) | set(range(448, 512))
    c.table = full
    sel = np.full((c.Tq, 1002), -1, np.int32)
    for t in range(c.Tq):
        b = 0 if t < 2 else 1
        keys = [p for p in (c.sel[t].tolist() if sparse else range(c.ctx[b])) if p >= 0 and (b or p not in bad)]
        sel[t, :len(keys)] = keys
    c.check(out, lse, ref=c.reference(sel=sel))
    # inconsistent lengths: sequence 0 has fewer keys than queries
    c = Case(62, [100, 300], [2, 1], 2, 4, 64, fmt, k=80 if sparse else None)
    ref = c.reference()
    c.lens[0] = 1
    out, lse = c.run(ctx)
    assert ctx.device_status() == 4
    c.check(out, lse, ref=ref, rows=[2])
    import torch
    assert torch.all(out[:2] == (0.0 if sparse else 77.0))
    if sparse:                                  # a position at the sequence's end
        c = Case(63, [100], [1], 1, 4, 64, fmt, masked=False, k=20)
        want = c.sel.copy()
        want[0, 7] = -1
        c.sel[0, 7] = 101
        out, lse = c.run(ctx)
        assert ctx.device_status() == 4
        c.check(out, lse, ref=c.reference(sel=want))


def test_strides_and_layouts(ctx):
    import torch
    c = Case(71, [300], [5], 2, 4, 128, A.BF16)
    d = c.device()
    packed = torch.randn((c.Tq, 2 * c.H, c.D), device="cuda").bfloat16()
    packed[:, c.H:] = d["q"]
    for q in (packed[:, c.H:], d["q"].transpose(0, 1).contiguous().transpose(0, 1)):
        for out in (torch.full((c.H, c.Tq, c.D), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1),
                    torch.full((c.Tq, c.H, c.D + 8), 3.0, dtype=torch.bfloat16, device="cuda")[:, :, :c.D]):
            o, lse = c.run(ctx, out=out, q=q, d=d)
            c.check(o, lse)
    # the same row for every token
    one = d["q"][:1].expand(c.Tq, -1, -1)
    c.q[:] = c.q[:1]
    c.check(*c.run(ctx, q=one, d=d))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("sparse", [False, True])
def test_no_writes_outside_buffers(ctx, fmt, sparse):
    import torch
    c = Case(81, [900, 20, 2000], [3, 1, 30], 2, 5, 128, fmt, k=70 if sparse else None)
    pad = 4096

    def padded(n):
        whole = torch.full((n + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
        return whole, whole[pad:pad + n]

    ow, o = padded(c.Tq * c.H * c.D * 2)
    lw, le = padded(c.Tq * c.H * 4)
    ww, ws = padded(ctx.attn_workspace_size(c.D))
    d = c.device()
    keep = d["cache"].clone()
    out, lse = c.run(ctx, out=o.view(torch.bfloat16).view(c.Tq, c.H, c.D), lse=le.view(torch.float32).view(c.Tq, c.H), ws=ws, d=d)
    c.check(out, lse)
    for w in (ow, lw, ww):
        assert torch.all(w[:pad] == 0x5A) and torch.all(w[-pad:] == 0x5A)
    assert torch.equal(d["cache"], keep)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("sparse", [False, True])
def test_repeats_streams_and_graphs_give_the_same_bits(ctx, fmt, sparse):
    import torch
    c = Case(91, [3000, 500], [4, 9], 2, 8, 128, fmt, k=300 if sparse else None)
    d = c.device()
    out, lse = c.run(ctx, d=d)
    c.check(out, lse)
    ws = torch.empty(ctx.attn_workspace_size(128), dtype=torch.uint8, device="cuda")
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
    d["q"].copy_(d["q"].roll(1, 0))
    g.replay()
    torch.cuda.synchronize()
    c.q = np.roll(c.q, 1, 0)
    c.check(o2, l2)
    assert ctx.device_status() == 0


def test_without_lse_and_without_queries(ctx):
    import torch
    c = Case(95, [50, 60], [2, 0], 1, 4, 64, A.FP8)
    d = c.device()
    out, lse = c.run(ctx, d=d)
    o2 = torch.empty_like(out)
    ws = torch.empty(ctx.attn_workspace_size(64), dtype=torch.uint8, device="cuda")
    ctx.tree_attn(d["q"], d["cache"], c.pages, c.fmt, 1, d["table"], d["lens"], d["cu"], o2, ws, mask=d["mask"])
    assert torch.equal(out, o2)
    ctx.tree_attn(d["q"][:0], d["cache"], c.pages, c.fmt, 1, d["table"][:1], d["lens"][1:], d["cu"][:2] * 0, o2[:0], ws)
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", [A.BF16, A.FP8, A.FP4])
def test_cache_past_32_bits(ctx, fmt):
    # a cache of more than 4 GB, the sequence's pages at its far end
    import torch
    from dsa_sparse_attention_store_gb300 import kv_page_bytes
    kv, D = 4, 128
    c = Case(99, [300], [2], kv, 2, D, fmt)
    pb = kv_page_bytes(kv, D, fmt)
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
    pos = torch.arange(302, dtype=torch.int32, device="cuda")
    k = torch.empty((302, kv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ctx.kv_load(big, shift + small, fmt, pos, torch.zeros_like(pos), d["table"], k, v)
    K, V = A.values(c.cache, small, kv, D, fmt)
    at = c.table[0, np.arange(302) // 64].astype(np.int64) * 64 + np.arange(302) % 64
    assert np.array_equal(k.double().cpu().numpy(), K[at]) and np.array_equal(v.double().cpu().numpy(), V[at])
    assert ctx.device_status() == 0


def test_binding_refusals(ctx):
    import torch
    from dsa_sparse_attention_store_gb300 import Rope, dsaidx
    c = Case(97, [50], [2], 1, 4, 64, A.BF16, k=16)
    d = c.device()
    out, lse = c.run(ctx, d=d)
    ws = torch.empty(ctx.attn_workspace_size(64), dtype=torch.uint8, device="cuda")

    def tree(**kw):
        a = dict(q=d["q"], cache=d["cache"], num_pages=c.pages, fmt=c.fmt, kv_heads=1, page_table=d["table"],
                 seq_lens=d["lens"], cu_q=d["cu"], out=out, workspace=ws, mask=d["mask"], lse=lse)
        a.update(kw)
        ctx.tree_attn(**a)

    tree()
    for kw, err in [(dict(q=d["q"].float()), TypeError), (dict(q=d["q"].cpu()), TypeError), (dict(q=d["q"][0]), ValueError),
                    (dict(out=out[:1]), ValueError), (dict(cache=d["cache"][:-1]), ValueError), (dict(cache=d["cache"].int()), TypeError),
                    (dict(lse=lse[:, :2]), ValueError), (dict(mask=d["mask"][:1]), ValueError), (dict(mask=d["mask"].long()), TypeError),
                    (dict(seq_lens=d["lens"].repeat(2)), ValueError), (dict(cu_q=d["cu"][:1]), ValueError), (dict(kv_heads=3), ValueError),
                    (dict(q=d["q"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError)]:
        with pytest.raises(err):
            tree(**kw)
    for kw, status in [(dict(workspace=ws[:-1]), 6), (dict(workspace=ws[1:]), 1), (dict(kv_heads=3, num_pages=1), 1), (dict(scale=0.0), 1),
                       (dict(q=torch.zeros((2, 4, 96), dtype=torch.bfloat16, device="cuda"),
                             out=torch.zeros((2, 4, 96), dtype=torch.bfloat16, device="cuda")), 2)]:
        with pytest.raises(dsaidx.DsaError) as e:
            tree(**kw)
        assert e.value.status == status, kw
    with pytest.raises(ValueError):
        ctx.sparse_attn(d["q"], d["sel"][:1], d["cache"], c.pages, c.fmt, 1, d["table"], d["lens"], d["cu"], out, ws)
    rope = Rope(ctx, rot_dim=64, max_pos=16)
    rope.close()
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ctx.kv_store(k, k, at, at, d["table"], d["cache"], c.pages, c.fmt, rope=rope)
    with pytest.raises(ValueError):
        ctx.rope_apply(k, at, rope)
    wide = Rope(ctx, rot_dim=64, max_pos=16)
    with pytest.raises(dsaidx.DsaError) as e:     # the rotated part passes the end of the head
        ctx.rope_apply(k, at, wide, rot_start=2)
    assert e.value.status == 1
    with pytest.raises(dsaidx.DsaError) as e:
        ctx.kv_store(k, k, at, at, d["table"], d["cache"], c.pages, c.fmt, rope=wide, rot_start=2)
    assert e.value.status == 1
    wide.close()
    with pytest.raises(dsaidx.DsaError) as e:     # a table that does not fit is refused and leaves no error behind
        Rope(ctx, rot_dim=1024, max_pos=2 ** 31 - 1)
    assert e.value.status == 3
    tree()
    torch.cuda.synchronize()
    assert ctx.device_status() == 0
