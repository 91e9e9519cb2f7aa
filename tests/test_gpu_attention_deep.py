"""Attention on the GPU where a thread block works through dozens of key tiles
and many units: rings wrap, units of one and of two row groups follow each
other. Against a 64-bit reference by torch (the definition, whole matrices);
every case runs twice and gives the same bits."""
import math

import numpy as np
import pytest

from oracle import attention as A
from tests.test_gpu_attention import Case

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


def _places(c, b, pos):
    """Rows of the flattened cache of sequence b's positions."""
    return c.table[b, pos // 64].astype(np.int64) * 64 + pos % 64


def reference(c):
    """As oracle.attention.attend, in whole matrices: (out, lse, sum w|v|,
    largest visible sum |q||k|) in 64 bits."""
    import torch
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    K, V = (up(x) for x in A.values(c.cache, c.pages, c.kv, c.D, c.fmt))
    q = up(c.q.astype(np.float64))
    out = torch.zeros((c.Tq, c.H, c.D), dtype=torch.float64, device="cuda")
    wabs, lse = torch.zeros_like(out), torch.full((c.Tq, c.H), -math.inf, dtype=torch.float64, device="cuda")
    qk = torch.zeros_like(lse)
    for b in range(c.B):
        n, r0, ctx_len = c.nds[b], int(c.cu[b]), c.ctx[b]
        if n == 0:
            continue
        if c.mask is None:
            tree = np.tril(np.ones((n, n), bool))
        else:
            tree = np.stack([A.visible(c.mask[r0 + i], n) for i in range(n)])
        new = _places(c, b, np.arange(ctx_len, ctx_len + n))
        for rows in [range(n)] if c.sel is None else [[i] for i in range(n)]:
            if c.sel is None:
                at = np.concatenate([_places(c, b, np.arange(ctx_len)), new])
                see = np.concatenate([np.ones((n, ctx_len), bool), tree], 1)
            else:
                pos = c.sel[r0 + rows[0]].astype(np.int64)
                pos = pos[pos >= 0]
                own = new[tree[rows[0]]] if c.mask is not None else new[:0]
                at = np.concatenate([_places(c, b, pos), own])
                see = np.ones((1, len(at)), bool)
            if len(at) == 0:
                continue
            at, hide = up(at), ~up(see).repeat_interleave(c.G, 0)[None]
            t = slice(r0 + rows[0], r0 + rows[0] + len(rows))
            m = len(rows)
            # [kv, rows x G, D] and [kv, keys, D]
            qq = q[t].view(m, c.kv, c.G, c.D).transpose(0, 1).reshape(c.kv, m * c.G, c.D)
            k, v = K[at].transpose(0, 1), V[at].transpose(0, 1)
            z = (qq @ k.transpose(1, 2) * c.scale).masked_fill_(hide, -math.inf)
            total = torch.logsumexp(z, -1, keepdim=True)
            w = torch.exp(z - torch.where(torch.isfinite(total), total, torch.zeros_like(total)))
            back = lambda x: x.view(c.kv, m, c.G, -1).transpose(0, 1).reshape(m, c.H, -1)  # noqa: E731
            out[t], wabs[t] = back(w @ v), back(w @ v.abs())
            lse[t] = back(total)[..., 0]
            qk[t] = back((qq.abs() @ k.abs().transpose(1, 2)).masked_fill_(hide, 0.0).amax(-1, keepdim=True))[..., 0]
    return tuple(x.cpu().numpy() for x in (out, lse, wabs, qk))


def check_twice(c, ctx, ref=None, rows=None):
    import torch
    d = c.device()
    out, lse = c.run(ctx, d=d)
    again, lse2 = c.run(ctx, d=d)
    assert ctx.device_status() == 0
    c.check(out, lse, ref=reference(c) if ref is None else ref, rows=rows)
    # as bits: NaN compares unequal to itself
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ctx_lens,nds,kv,G,D,masked", [
    # units of 256 and 128 rows, of 31 tiles whose last holds one key
    ([1873] * 16, [48] * 16, 8, 8, 128, True),
    # units of 256 and 64 rows
    ([1930] * 24, [20] * 24, 8, 16, 64, True),
    # decode steps of about 3000 keys and, among them, chunks of a prefill
    ([x for i in range(8) for x in (3000 + 70 * i, 3400 - 30 * i, 2900 + i, 700 + 50 * i)], [1, 1, 1, 150 + 9] * 8, 8, 8, 64, False),
])
def test_short_units_before_long_ones(ctx, fmt, ctx_lens, nds, kv, G, D, masked):
    # the second group of rows has nothing to do in units of at most 128 rows
    # and is far ahead of the loaders when the next unit starts
    check_twice(Case(len(nds), ctx_lens, nds, kv, G, D, fmt, masked=masked), ctx)


def _poison(c, b, j):
    """Drafted token j of sequence b has values that are NaN in the first 32 dimensions of every kv head."""
    _, _, vc, vs = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)
    pos = c.ctx[b] + j
    p, o = c.table[b, pos // 64], pos % 64
    if c.fmt == A.BF16:
        vc.view(np.uint16)[p, :, o, :32] = 0x7FC1
    else:
        vs[p, :, o, 0] = 255


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_runs_of_one_tile_units(ctx, fmt, D):
    # per kv head 13 units of a long sequence, then runs of 160 units of one
    # tile and 16 rows, in which the second group has nothing to do. What it
    # still has to learn about its last unit must not be overwritten meanwhile.
    ctx_lens, nds = [], []
    for i in range(12):
        ctx_lens += [90 + 17 * i] + [(5 * j + i) % 60 for j in range(20)]
        nds += [200] + [1] * 20
    c = Case(5 + D, ctx_lens, nds, 8, 16, D, fmt)
    bits = c.bits.copy()
    big = [b for b, n in enumerate(nds) if n == 200]
    for b in big:                               # its last token is seen by itself and token 150 alone
        bits[c.cu[b]:c.cu[b + 1], 199] = False
        bits[c.cu[b] + 199, 199] = bits[c.cu[b] + 150, 199] = True
    c.set_bits(bits)
    clean = reference(c)
    check_twice(c, ctx, clean)
    for b in big:
        _poison(c, b, 199)
    hit = sorted(int(c.cu[b]) + i for b in big for i in (150, 199))
    rows = [t for t in range(c.Tq) if t not in set(hit)]
    check_twice(c, ctx, clean, rows)
    out, _ = c.run(ctx)
    got, want = out.double().cpu().numpy()[hit], clean[0][hit]
    assert np.all(np.isnan(got[..., :32])) and np.all(np.isfinite(got[..., 32:]))
    tol = A.tolerance(*clean, c.scale, D, float(c.lens.max()))[0][hit]
    assert np.all(np.abs(got - want)[..., 32:] <= tol[..., 32:])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nd,G", [(9, 3), (19, 5), (70, 4)])   # 27, 95 and 280 rows: each form, warps that are not full
def test_rows_that_see_different_replaced_values(ctx, fmt, D, nd, G):
    # a third of the drafted tokens, on both sides of a page's end, hold what is
    # not finite; every row sees others of them, some none
    c = Case(77 + nd, [50], [nd], 2, G, D, fmt)
    rng = np.random.default_rng(nd + D)
    bits = np.zeros_like(c.bits)
    bits[:, :nd] = rng.random((nd, nd)) < rng.choice([0.0, 0.1, 0.5], (nd, 1))
    c.set_bits(bits)
    clean = c.reference()
    _, _, vc, vs = A.fields(c.cache, c.pages, c.kv, D, fmt)
    for j in rng.permutation(nd)[:nd // 3]:
        pos = 50 + int(j)
        p, o = c.table[0, pos // 64], pos % 64
        for h in range(c.kv):
            if fmt == A.BF16:
                d = rng.permutation(D)[:9]
                vc.view(np.uint16)[p, h, o, d] = rng.choice([0x7FC1, 0x7F80, 0xFF80], 9)
            else:
                vs[p, h, o, rng.integers(D // 32)] = 255
    o, z, _, _ = c.reference()
    assert np.isnan(o).any() and np.isfinite(o).all(axis=(1, 2)).any()
    out, lse = c.run(ctx)
    assert ctx.device_status() == 0
    got = out.double().cpu().numpy()
    for kind in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(kind(got), kind(o)), kind
    fin = np.isfinite(o)
    tol, tol_lse = A.tolerance(*clean, c.scale, D, float(c.lens.max()))
    assert np.all(np.abs(got - clean[0])[fin] <= tol[fin])
    assert np.all(np.abs(lse.double().cpu().numpy() - clean[1]) <= tol_lse)


# sequences of about so many key tiles: on both sides of what the rings hold
TILES = [1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64]
FORMS = [  # new tokens, kv heads, G, keys selected (0: the tree form): up to 32, up to 128 and more rows
    (2, 8, 4, 0), (8, 8, 8, 0), (20, 4, 16, 0), (5, 8, 4, 700), (3, 8, 40, 1100)]


def _deep(seed, form, fmt, D, copies, masked=True, **kw):
    nd, kv, G, k = form
    tiles = TILES * copies
    return Case(seed, [max(0, 64 * t - nd - (i % 3)) for i, t in enumerate(tiles)], [nd] * len(tiles), kv, G, D, fmt, masked=masked,
                k=k or None, **kw)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,masked", [(64, False), (128, True)])
@pytest.mark.parametrize("form", FORMS)
def test_dozens_of_tiles_a_block(ctx, fmt, D, form, masked):
    check_twice(_deep(7, form, fmt, D, 3 if form[3] == 0 else 2, masked), ctx)


def _rise(c):
    """Keys grow by a power of two every other page of a sequence."""
    kc, ks, _, _ = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)
    for b in range(c.B):
        for j in range(-(-int(c.lens[b]) // 64)):
            e, p = min(j // 2, 6), c.table[b, j]
            if c.fmt == A.BF16:
                w = kc[p].view(np.uint16)
                w[...] = np.where(w & 0x7F80, w + (e << 7), w)
            else:
                ks[p] += e


def _jumps(c, b):
    """Of sequence b's rows of kv head 0, the share whose running maximum, in
    tiles of 64 keys in the order the kernel takes them, rises by more than 2^8
    after the first tile that holds a key."""
    K, _ = A.values(c.cache, c.pages, c.kv, c.D, c.fmt)
    hits, rows = 0, 0
    for i in range(c.nds[b]):
        t = int(c.cu[b]) + i
        pos = c.sel[t][c.sel[t] >= 0] if c.sel is not None else np.arange(c.ctx[b])
        s = c.q[t, :c.G].astype(np.float64) @ K[_places(c, b, pos), 0].T * c.scale / math.log(2)
        top = np.stack([s[:, x:x + 64].max(1) for x in range(0, s.shape[1], 64)], 1)
        run = np.maximum.accumulate(top, 1)
        hits += int((np.diff(run, axis=1) > 8).any(1).sum())
        rows += c.G
    return hits / rows


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_maximum_moves_in_later_tiles(ctx, fmt, D, form):
    # the accumulator and the sums are rescaled between products
    c = _deep(8, form, fmt, D, 2, q_gain=2.0)
    _rise(c)
    if c.sel is not None:
        for t in range(c.Tq):                   # ascending positions, and a first tile without a key for every third query
            s = np.sort(c.sel[t][c.sel[t] >= 0])
            c.sel[t] = -1
            at = 64 if t % 3 == 0 and len(s) + 64 <= c.sel.shape[1] else 0
            c.sel[t, at:at + len(s)] = s
    assert _jumps(c, len(TILES) - 1) > 0.5 and _jumps(c, len(TILES) - 4) > 0.5
    check_twice(c, ctx)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nd,G", [(110, 1), (150, 2)])
def test_first_tile_hidden_from_some_rows(ctx, fmt, D, nd, G):
    # no committed context: half of the rows see nothing of the first tile (or
    # two), which others do, and their maximum begins later
    c = Case(9, [0] * 40, [nd] * 40, 8, G, D, fmt, q_gain=2.0)
    bits = c.bits.copy()
    for b in range(40):
        for i in range(0, nd, 2):
            bits[c.cu[b] + i, :64 + 64 * (b % 2 if nd > 128 else 0)] = False
            bits[c.cu[b] + i, nd - 1 - b % 7] = True
    c.set_bits(bits)
    _rise(c)
    check_twice(c, ctx)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("steps,chunk,kv,G,D", [
    (63, 1100, 2, 8, 128),      # the mean chooses 256 rows: the steps have 8 of them
    (255, 512, 1, 8, 64),       # the mean chooses 32 rows: the chunk is 128 units
    (40, 300, 2, 12, 64),       # the mean chooses 128 rows
])
def test_decode_steps_beside_a_chunk(ctx, fmt, steps, chunk, kv, G, D):
    # a serving batch: one chunk of a prefill among decode steps, no mask
    ctx_lens, nds = [(97 * i) % 1500 for i in range(steps)], [1] * steps
    ctx_lens.insert(steps // 3, 700)
    nds.insert(steps // 3, chunk)
    check_twice(Case(steps, ctx_lens, nds, kv, G, D, fmt, masked=False), ctx)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ctx_lens,nds,kv,G", [
    ([0], [1500], 1, 64),                       # 375 row tiles of four tokens
    ([100, 64, 3], [700, 513, 1], 2, 40),       # a token ends inside a row tile
    ([0, 63, 2000, 5], [400, 0, 900, 64], 3, 1),    # 256 tokens a row tile
    ([31, 0, 65], [257, 255, 256], 1, 7),
])
def test_chunks_of_many_row_tiles(ctx, fmt, ctx_lens, nds, kv, G):
    # the plan counts row tiles by their number of key tiles; cuts fall anywhere in them
    check_twice(Case(3 + G, ctx_lens, nds, kv, G, 64, fmt, masked=False), ctx)
