"""A step's page tables and slot maps on the GPU against the reference, value
for value: sequences that grow, start, rest and end, pools that run short or
over, lengths and pages out of range, padded batches, graphs, and the pages'
whole life over many steps."""
import numpy as np
import pytest

from oracle import spans as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import torch
    from dsa_sparse_attention_store_gb300 import Context
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    c = Context(max_pos=64)
    yield c
    c.close()


def _pool(rng, old, width, spare, extra=0):
    """A table whose rows have pages for `old` tokens, and a stack of `spare` more."""
    pages = [min(width, -(-max(o, 0) // 64)) for o in old]
    n = sum(pages) + spare
    order = rng.permutation(n + extra).astype(np.int32)
    table = rng.integers(-5, n, (len(old), width)).astype(np.int32)      # what lies past a row's pages does not matter
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    stack = np.full(n + extra, -7, np.int32)
    stack[:spare] = order[at:at + spare]
    return table, stack, n + extra


def _run(ctx, old, new, table, num_pages, stack, count, T, own_from=None, slots=True, keep=None):
    import torch
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    B = len(old)
    fresh = lambda n: torch.full((n,), 99, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dict(old=d(old), new=d(new), table=d(table), stack=d(stack), count=d([count]), left=fresh(1), lens=fresh(B), cu=fresh(B + 1),
             seq=fresh(T), pos=fresh(T), slot=fresh(T) if slots else None, own=None if own_from is None else d(own_from))
    go = lambda: ctx.batch_plan(t["old"], t["new"], t["table"], num_pages, t["stack"], t["count"], t["left"], t["lens"], t["cu"],  # noqa: E731
                                t["seq"], t["pos"], t["slot"], own_from=t["own"])
    go()
    if keep is not None:
        keep.update(t, go=go)
    return t


def _check(ctx, t, want):
    assert ctx.device_status() == (4 if want["bad"] else 0)
    for k in ("table", "stack", "lens", "cu", "seq", "pos", "slot"):
        if t[k] is not None:
            got = t[k].cpu().numpy()
            assert np.array_equal(got, want[k]), (k, np.argwhere(got != want[k])[:5].tolist())
    assert int(t["left"]) == want["left"]


def _case(ctx, rng, old, new, width, spare, T=None, own_from=None, extra=0, num_pages=None, count=None, **kw):
    table, stack, n = _pool(rng, old, width, spare, extra)
    T = sum(max(x, 0) for x in new) if T is None else T
    args = (old, new, table, n if num_pages is None else num_pages, stack, spare if count is None else count, T, own_from)
    want = S.batch_plan(*args)
    t = _run(ctx, *args, **kw)
    _check(ctx, t, want)
    return t, want


@pytest.mark.parametrize("B,most,ends", [(1, 1, False), (1, 300, False), (5, 70, True), (64, 1, False), (64, 200, True), (1000, 9, True),
                                         (1025, 1, False), (2500, 40, True)])
@pytest.mark.parametrize("seed", range(3))
def test_plan_matches_reference(ctx, B, most, ends, seed):
    rng = np.random.default_rng([B, most, seed])
    old = rng.integers(0, 700, B)
    new = rng.integers(0, most + 1, B)
    if ends:
        new[rng.random(B) < 0.3] = -1
    own = rng.integers(0, 4, B) if seed == 2 else None
    need = int(sum(-(-(o + n) // 64) - -(-o // 64) for o, n in zip(old, new) if n >= 0))
    _case(ctx, rng, old, new, 16, need + seed, own_from=own, T=int(new.clip(0).sum()) + [0, 1, 900][seed], slots=seed != 1)


@pytest.mark.parametrize("B,most", [(300, 9000), (4095, 40), (8192, 3), (8193, 3), (16384, 40), (16385, 3), (40002, 12)])
@pytest.mark.parametrize("shift", [0, 1])             # whether four tokens are one store
def test_many_sequences_and_tokens(ctx, B, most, shift):
    import torch
    rng = np.random.default_rng([B, shift])
    old = rng.integers(0, 200, B)
    new = rng.integers(0, most, B)
    new[rng.random(B) < 0.2] = -1
    new[-3:] = [7, -1, 5]
    own = rng.integers(0, 3, B)
    width = -(-(200 + most) // 64)
    table, stack, pages = _pool(rng, old, width, 30000)
    T = int(new.clip(0).sum()) + 101
    t = {}
    _run(ctx, old, new, table, pages, stack, 30000, T, own, keep=t)
    if shift:
        for k, v in (("table", table), ("stack", stack)):
            t[k].copy_(torch.from_numpy(v))
        for k in ("seq", "pos", "slot"):
            t[k] = torch.full((T + 1,), 99, dtype=torch.int32, device="cuda")[1:]
        ctx.batch_plan(t["old"], t["new"], t["table"], pages, t["stack"], t["count"], t["left"], t["lens"], t["cu"],
                       t["seq"], t["pos"], t["slot"], own_from=t["own"])
    _check(ctx, t, S.batch_plan(old, new, table, pages, stack, 30000, T, own))


def test_lengths_around_pages(ctx):
    rng = np.random.default_rng(1)
    old = [o for o in (0, 1, 63, 64, 65, 127, 128) for _ in range(6)]
    new = [n for _ in range(7) for n in (0, 1, 63, 64, 65, 200)]
    _case(ctx, rng, old, new, 6, 200)
    _case(ctx, rng, old, [0] * 42, 6, 0)                   # nothing to do
    _case(ctx, rng, old, [-1] * 42, 6, 3)                  # all of them end
    _case(ctx, rng, [0] * 42, new, 6, 200)                 # all of them start


def test_pages_that_come_back_are_used_first(ctx):
    # more taken than returned, as many, fewer; the free stack touched only for the rest
    rng = np.random.default_rng(2)
    for new in ([-1, 320, -1, 64], [-1, 192, -1, 64], [-1, 64, -1, 64]):
        t, want = _case(ctx, rng, [128, 0, 100, 0], new, 8, 9)
        assert not want["bad"]


def test_too_few_pages(ctx):
    rng = np.random.default_rng(3)
    t, want = _case(ctx, rng, [10, 64, 0, 90, 0], [60, 64, 130, 100, 1], 5, 3)
    assert want["bad"] and want["left"] == 0 and (want["slot"] == -1).any()
    _case(ctx, rng, [0, 0], [64, 64], 3, 0, num_pages=1)    # none at all (a cache has at least one)


def test_out_of_range(ctx):
    rng = np.random.default_rng(4)
    # negative and too long lengths, a length of the table's width, a negative own_from
    _case(ctx, rng, [-1, 100, 300, 320, 2 ** 31 - 1, 64], [5, 300, 20, 0, 2 ** 31 - 1, 256], 5, 40, T=600)
    _case(ctx, rng, [70, 100], [-1, 3], 5, 4, own_from=[-1, 0])
    _case(ctx, rng, [70, 100], [-1, 3], 5, 4, own_from=[99, 0])          # nothing of its own: no page comes back
    # more tokens than the maps have places for: the pages are taken all the same
    _case(ctx, rng, [0, 10], [200, 100], 5, 9, T=150)
    # page ids that the cache does not have
    _case(ctx, rng, [100, 70, 30], [100, 3, 40], 5, 9, num_pages=6)
    # a count that is not one; a stack that cannot take what comes back
    for count in (-3, 12, 2 ** 31 - 1):
        _case(ctx, rng, [100, 0], [-1, 64], 5, 9, count=count)
    table, stack, n = _pool(rng, [640, 0], 10, 2)
    args = ([640, 0], [-1, 1], table, n, stack[:4], 2, 1, None)
    _check(ctx, _run(ctx, *args), S.batch_plan(*args))


@pytest.mark.parametrize("B", [3, 3000])
def test_again_on_a_stream_and_in_a_graph(ctx, B):
    # inputs are only read: the same call gives the same; a replay sees other lengths
    import torch
    rng = np.random.default_rng(5)
    old, new = rng.integers(0, 300, B), rng.integers(-1, 90, B)
    keep = {}
    t, want = _case(ctx, rng, old, new, 8, 3 * B, T=90 * B, keep=keep)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        keep["go"]()
        keep["go"]()
    s.synchronize()
    _check(ctx, t, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        keep["go"]()
    table, stack = t["table"].cpu().numpy(), t["stack"].cpu().numpy()
    again = np.where(new < 0, -1, rng.integers(0, 60, B))
    t["new"].copy_(torch.from_numpy(again.astype(np.int32)))
    g.replay()
    torch.cuda.synchronize()
    want = S.batch_plan(old, again, table, len(stack), stack, 3 * B, 90 * B)
    _check(ctx, t, want)


def test_no_writes_outside_buffers(ctx):
    import torch
    rng = np.random.default_rng(6)
    old, new = [100, 70, 0], [30, -1, 64]
    table, stack, n = _pool(rng, old, 4, 5)
    want = S.batch_plan(old, new, table, n, stack, 5, 100)
    sizes = dict(table=12, stack=len(stack), left=1, lens=3, cu=4, seq=100, pos=100, slot=100)
    whole = {k: torch.full((m + 128,), 123456, dtype=torch.int32, device="cuda") for k, m in sizes.items()}
    part = {k: whole[k][64:64 + m] for k, m in sizes.items()}
    part["table"].copy_(torch.from_numpy(table).flatten())
    part["stack"].copy_(torch.from_numpy(stack))
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx.batch_plan(d(old), d(new), part["table"].view(3, 4), n, part["stack"], d([5]), part["left"], part["lens"], part["cu"],
                   part["seq"], part["pos"], part["slot"])
    part["table"] = part["table"].view(3, 4)
    _check(ctx, part, want)
    for k, m in sizes.items():
        assert torch.all(whole[k][:64] == 123456) and torch.all(whole[k][64 + m:] == 123456), k


def test_a_pool_over_many_steps(ctx):
    # sequences come, grow and go; no page is ever in two places, none is lost
    rng = np.random.default_rng(7)
    B, width, n, T = 40, 12, 300, 40 * 150
    table, stack, old, left = np.full((B, width), -1, np.int32), np.arange(n, dtype=np.int32), np.zeros(B, np.int32), n
    for step in range(30):
        new = np.where(old == 0, rng.integers(0, 150, B), rng.integers(1, 20, B))
        new[(old + new > 700) | ((old > 0) & (rng.random(B) < 0.1))] = -1
        args = (old, new, table, n, stack, left, T)
        t, want = _run(ctx, *args), S.batch_plan(*args)
        _check(ctx, t, want)
        assert not want["bad"]
        table, stack, left, old = t["table"].cpu().numpy(), t["stack"].cpu().numpy(), int(t["left"]), t["lens"].cpu().numpy()
        used = [p for b in range(B) for p in table[b, :-(-old[b] // 64)]]
        assert sorted(used + stack[:left].tolist()) == list(range(n))


def test_refusals(ctx):
    import torch
    from dsa_sparse_attention_store_gb300 import dsaidx
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    a = dict(old_lens=i32(2), new_lens=i32(2), page_table=i32(2, 3), num_pages=9, free_pages=i32(9), free_count=i32(1), free_left=i32(1),
             seq_lens=i32(2), cu_q=i32(3), seq_id=i32(5), cache_pos=i32(5), slots=i32(5))
    ctx.batch_plan(**a)
    for k, v, err in [("old_lens", i32(3), ValueError), ("new_lens", i32(2).long(), TypeError), ("cu_q", i32(2), ValueError),
                      ("slots", i32(4), ValueError), ("own_from", i32(1), ValueError), ("page_table", i32(3, 2).t(), ValueError),
                      ("free_count", i32(2), ValueError), ("free_pages", i32(9).cpu(), TypeError)]:
        with pytest.raises(err):
            ctx.batch_plan(**dict(a, **{k: v}))
    for kw in (dict(seq_lens=a["old_lens"]), dict(free_left=a["free_count"]), dict(cache_pos=a["seq_id"]), dict(slots=a["seq_id"]),
               dict(free_pages=a["page_table"].view(-1)), dict(seq_lens=a["cu_q"][1:])):
        with pytest.raises(dsaidx.DsaError) as e:
            ctx.batch_plan(**dict(a, **kw))
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert ctx.device_status() == 0
