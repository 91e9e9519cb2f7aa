"""Rotary positions and the K/V cache on the GPU against the 64-bit reference:
layouts, parts, scalings, types, strides, alignments, both directions; stored
bytes of every format, reading back, and what is out of range."""
import numpy as np
import pytest

from oracle import attention as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import torch
    from dsa_sparse_attention_store_gb300 import Context
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    c = Context(max_pos=64)
    yield c
    c.close()


def _rope(ctx, rot, max_pos=4096, **kw):
    from dsa_sparse_attention_store_gb300 import Rope
    return Rope(ctx, rot_dim=rot, max_pos=max_pos, **kw)


def _types():
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# half a step of the type, and of an fp32 product and sum (three roundings of
# values no larger than |a| + |b|, and the table's two): the bounds count those
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def _check_rope(got, x, want, dtype, mscale=1.0):
    mag = np.abs(x).max(axis=-1, keepdims=True) * 2 * mscale
    tol = np.abs(want) * HALF[dtype] * 1.001 + mag * 5 * 2.0 ** -24 + (2.0 ** -24 if dtype == "fp16" else 1e-38)
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot,start", [(1, 1, 128, 128, 0), (7, 3, 128, 64, 64), (33, 5, 80, 20, 0), (5, 2, 81, 6, 3),
                                             (2, 64, 64, 32, 32), (130, 9, 192, 64, 128), (3, 1, 2, 2, 0), (4, 40, 100, 48, 52)])
def test_rope_matches_reference(ctx, dtype, layout, T, H, D, rot, start):
    import torch
    g = torch.Generator().manual_seed(T * 1000 + D)
    x = torch.randn((T, H, D), generator=g).to(_types()[dtype])
    pos = torch.randint(0, 4096, (T,), generator=g, dtype=torch.int32)
    rope = _rope(ctx, rot, layout=layout)
    for inverse in (False, True):
        out = torch.full_like(x.cuda(), 9.0)
        ctx.rope_apply(x.cuda(), pos.cuda(), rope, out=out, rot_start=start, inverse=inverse)
        want = A.rope(x.double().numpy(), pos.numpy(), rot, start, layout, A.frequencies(rot), inverse=inverse)
        _check_rope(out.double().cpu().numpy(), x.double().numpy(), want, dtype)
        same = x.cuda()
        ctx.rope_apply(same, pos.cuda(), rope, rot_start=start, inverse=inverse)
        assert torch.equal(same, out)
    assert ctx.device_status() == 0
    rope.close()


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=8.0)),
                                        ("by_parts", dict(factor=4.0, orig_max_pos=4096, beta_slow=1.0, beta_fast=32.0)),
                                        ("by_parts", dict(factor=16.0, orig_max_pos=8192, beta_slow=0.5, beta_fast=20.0))])
def test_rope_scalings_at_far_positions(ctx, scaling, kw):
    import torch
    T, H, D, rot = 200, 2, 128, 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, H, D), generator=g)
    pos = torch.randint(130000, 131072, (T,), generator=g, dtype=torch.int32)
    rope = _rope(ctx, rot, max_pos=131072, scaling=scaling, mscale=1.25, theta=500000.0, **kw)
    y = torch.empty_like(x, device="cuda")
    ctx.rope_apply(x.cuda(), pos.cuda(), rope, out=y)
    f = A.frequencies(rot, 500000.0, scaling, kw["factor"], kw.get("orig_max_pos", 1), kw.get("beta_slow", 0), kw.get("beta_fast", 1))
    _check_rope(y.double().cpu().numpy(), x.double().numpy(), A.rope(x.double().numpy(), pos.numpy(), rot, 0, "half", f, 1.25), "fp32", 1.25)
    rope.close()


def test_rope_large_batch_takes_four_heads_a_thread(ctx):
    import torch
    T, H, D, rot = 3000, 37, 128, 64   # enough threads for the four-head form; heads not a multiple of four
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, H, D), generator=g, device="cuda").bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope = _rope(ctx, rot, layout="interleaved")
    y = torch.empty_like(x)
    ctx.rope_apply(x, pos, rope, out=y, rot_start=64)
    xn = x.double().cpu().numpy()
    _check_rope(y.double().cpu().numpy(), xn, A.rope(xn, np.arange(T), rot, 64, "interleaved", A.frequencies(rot)), "bf16")
    # and back: the inverse undoes it to two roundings
    ctx.rope_apply(y, pos, rope, rot_start=64, inverse=True)
    assert float((y.double() - x.double()).abs().max()) <= 2 * 2.0 ** -8 * float(x.abs().max()) * 1.5
    rope.close()


def test_rope_inverse_is_the_gradient(ctx):
    import torch
    T, H, D, rot, start = 9, 2, 32, 16, 8
    g = torch.Generator().manual_seed(8)
    x = torch.randn((T, H, D), generator=g)
    dy = torch.randn((T, H, D), generator=g)
    pos = torch.randint(0, 64, (T,), generator=g, dtype=torch.int32)
    rope = _rope(ctx, rot, mscale=1.5)
    dx = torch.empty_like(dy, device="cuda")
    ctx.rope_apply(dy.cuda(), pos.cuda(), rope, out=dx, rot_start=start, inverse=True)
    f = A.frequencies(rot)
    h = 1e-6
    xn, dyn = x.double().numpy(), dy.double().numpy()
    loss = lambda v: float((A.rope(v, pos.numpy(), rot, start, "half", f, 1.5) * dyn).sum())  # noqa: E731
    for (t, hd, d) in [(0, 0, 8), (3, 1, 15), (8, 0, 23), (4, 1, 31), (2, 0, 0), (5, 1, 16)]:
        up, dn = xn.copy(), xn.copy()
        up[t, hd, d] += h
        dn[t, hd, d] -= h
        assert abs((loss(up) - loss(dn)) / (2 * h) - float(dx[t, hd, d])) < 1e-5
    rope.close()


def test_rope_strides_alignment_and_range(ctx):
    import torch
    T, H, D, rot = 11, 4, 64, 32
    g = torch.Generator().manual_seed(9)
    rope = _rope(ctx, rot, max_pos=100)
    f = A.frequencies(rot)
    pos = torch.arange(T, dtype=torch.int32)
    for make in (lambda: torch.randn((H, T, D), generator=g).bfloat16().cuda().transpose(0, 1),       # heads outermost
                 lambda: torch.randn((T, H, D + 3), generator=g).bfloat16().cuda()[:, :, 1:1 + D],      # odd strides, misaligned
                 lambda: torch.randn((T, 3 * H, D), generator=g).bfloat16().cuda()[:, H:2 * H]):        # a slice of packed heads
        x = make()
        y = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        ctx.rope_apply(x, pos.cuda(), rope, out=y)
        xn = x.double().cpu().numpy()
        _check_rope(y.double().cpu().numpy(), xn, A.rope(xn, pos.numpy(), rot, 0, "half", f), "bf16")
        ctx.rope_apply(x, pos.cuda(), rope)
        assert torch.equal(x, y)
    assert ctx.device_status() == 0
    bad = pos.clone()
    bad[3], bad[7] = 100, -1
    x = torch.randn((T, H, D), generator=g).bfloat16().cuda()
    y = torch.full_like(x, 7.0)
    ctx.rope_apply(x, bad.cuda(), rope, out=y)
    assert ctx.device_status() == 4
    assert torch.all(y[3] == 7.0) and torch.all(y[7] == 7.0) and not torch.any(torch.all(y[4] == 7.0))
    rope.close()


# ------------------------------------------------------------------ cache

def _paged(rng, lens):
    pages = [max(1, -(-n // 64)) for n in lens]
    total = sum(pages) + 2
    order = rng.permutation(total)[:sum(pages)]
    table = np.full((len(lens), max(pages) + 1), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _inputs(rng, T, kv, D, big=True):
    k = rng.standard_normal((T, kv, D)).astype(np.float32)
    v = rng.standard_normal((T, kv, D)).astype(np.float32)
    if big:  # blocks of very different magnitudes, zeros, the type's extremes
        k *= np.exp2(rng.integers(-20, 20, (T, kv, 1))).astype(np.float32)
        v[0] = 0
        v[T // 2, 0, :32] = 3.3895313892515355e38
        v[T // 2, 0, 32:64] = 1e-38
        v[-1, -1, 1] = -448.0
    return k, v


@pytest.mark.parametrize("fmt", [A.BF16, A.FP8, A.FP4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,kv", [(1, 1), (5, 3), (131, 8)])
def test_store_bytes_and_load_match_reference(ctx, fmt, D, T, kv):
    import torch
    from dsa_sparse_attention_store_gb300 import kv_page_bytes
    rng = np.random.default_rng(100 * fmt + D + T)
    B = 3
    lens = [T + 70, 1, 200]
    table, pages = _paged(rng, lens)
    seq = np.zeros(T, np.int32)
    pos = (np.arange(T) + 60).astype(np.int32)
    if T > 1:
        seq[T // 2:] = 2
    k, v = _inputs(rng, T, kv, D)
    kb, vb = A.bf16_bits(k), A.bf16_bits(v)
    kt, vt = (torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() for x in (kb, vb))
    assert kv_page_bytes(kv, D, fmt) == kv * A.head_bytes(fmt, D)
    cache = torch.full((pages * kv_page_bytes(kv, D, fmt),), 0xA5, dtype=torch.uint8, device="cuda")
    dt = torch.from_numpy(table).cuda()
    ctx.kv_store(kt, vt, torch.from_numpy(pos).cuda(), torch.from_numpy(seq).cuda(), dt, cache, pages, fmt)
    assert ctx.device_status() == 0
    want = np.full(cache.numel(), 0xA5, np.uint8)
    kc, ks, vc, vs = A.fields(want, pages, kv, D, fmt)
    for t in range(T):
        p, o = table[seq[t], pos[t] // 64], pos[t] % 64
        for h in range(kv):
            kc[p, h, o], ks[p, h, o] = A.quantise(A.bf16_value(kb[t, h]), fmt)
            vc[p, h, o], vs[p, h, o] = A.quantise(A.bf16_value(vb[t, h]), fmt)
    assert np.array_equal(cache.cpu().numpy(), want)
    ko, vo = torch.full_like(kt, 5.0), torch.full_like(vt, 5.0)
    ctx.kv_load(cache, pages, fmt, torch.from_numpy(pos).cuda(), torch.from_numpy(seq).cuda(), dt, ko, vo)
    K, V = A.values(want, pages, kv, D, fmt)
    at = table[seq, pos // 64].astype(np.int64) * 64 + pos % 64
    assert np.array_equal(ko.double().cpu().numpy(), K[at]) and np.array_equal(vo.double().cpu().numpy(), V[at])
    assert ctx.device_status() == 0
    assert B == table.shape[0]


@pytest.mark.parametrize("fmt", [A.FP8, A.FP4])
def test_every_code_and_scale_reads_back(ctx, fmt):
    import torch
    D, kv = 128, 1
    cache = np.zeros(4 * A.head_bytes(fmt, D), np.uint8)
    kc, ks, vc, vs = A.fields(cache, 4, kv, D, fmt)
    codes = np.arange(256, dtype=np.uint8)
    if fmt == A.FP8:
        codes = codes[(codes & 0x7F) != 0x7F]      # the NaN codes are never written
    row = np.resize(codes, kc.shape[-1] * 4).reshape(4, -1)
    scales = np.arange(10, 247, dtype=np.uint8) if fmt == A.FP8 else np.arange(2, 253, dtype=np.uint8)
    for x in range(256):
        kc[x // 64, 0, x % 64] = row[x % 4]
        ks[x // 64, 0, x % 64] = scales[x % len(scales)]
        vc[x // 64, 0, x % 64] = row[(x + 1) % 4]
        vs[x // 64, 0, x % 64] = 255 if x == 9 else scales[(x * 7) % len(scales)]
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    pos = torch.arange(256, dtype=torch.int32, device="cuda")
    k = torch.empty((256, 1, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ctx.kv_load(torch.from_numpy(cache).cuda(), 4, fmt, pos, torch.zeros_like(pos), table, k, v)
    K, V = A.values(cache, 4, kv, D, fmt)
    assert np.array_equal(k.double().cpu().numpy(), K)
    assert np.array_equal(v.double().cpu().numpy(), V, equal_nan=True)


@pytest.mark.parametrize("fmt", [A.BF16, A.FP8, A.FP4])
@pytest.mark.parametrize("layout,rot,start", [("half", 64, 0), ("half", 32, 32), ("interleaved", 64, 0), ("interleaved", 24, 8),
                                              ("half", 20, 4), ("interleaved", 10, 3), ("half", 2, 62)])
def test_store_rotates_keys(ctx, fmt, layout, rot, start):
    import torch
    D, kv, T = 64, 2, 37
    rng = np.random.default_rng(rot + start)
    table, pages = _paged(rng, [T + 3])
    k, v = _inputs(rng, T, kv, D, big=False)
    kt, vt = torch.from_numpy(k).bfloat16().cuda(), torch.from_numpy(v).bfloat16().cuda()
    pos = torch.arange(3, T + 3, dtype=torch.int32, device="cuda")
    rpos = torch.from_numpy(rng.integers(0, 4096, T).astype(np.int32)).cuda()
    seq = torch.zeros_like(pos)
    rope = _rope(ctx, rot, layout=layout)
    cache = torch.zeros(pages * kv * A.head_bytes(fmt, D), dtype=torch.uint8, device="cuda")
    ctx.kv_store(kt, vt, pos, seq, torch.from_numpy(table).cuda(), cache, pages, fmt, rope=rope, rope_pos=rpos, rot_start=start)
    assert ctx.device_status() == 0
    # the rotation alone, in fp32, then the format: the same bytes
    y = kt.float()
    ctx.rope_apply(y, rpos, rope, rot_start=start)
    want = np.zeros(cache.numel(), np.uint8)
    kc, ks, vc, vs = A.fields(want, pages, kv, D, fmt)
    yn, vn = y.cpu().numpy(), vt.float().cpu().numpy()
    for t in range(T):
        p, o = table[0, (t + 3) // 64], (t + 3) % 64
        for h in range(kv):
            kc[p, h, o], ks[p, h, o] = A.quantise(yn[t, h], fmt)
            vc[p, h, o], vs[p, h, o] = A.quantise(vn[t, h], fmt)
    assert np.array_equal(cache.cpu().numpy(), want)
    rope.close()


def test_store_and_load_strides_range_and_nonfinite(ctx):
    import torch
    rng = np.random.default_rng(4)
    D, kv, T = 128, 4, 6
    table, pages = _paged(rng, [64, 64])
    table[1, 0] = pages + 5                      # a page out of range
    packed = torch.randn((T, 3 * kv, D), device="cuda").bfloat16()
    packed[0, kv, 3] = float("nan")
    packed[1, kv, 40] = float("inf")
    k, v = packed[:, kv:2 * kv], packed[:, 2 * kv:].transpose(0, 1).contiguous().transpose(0, 1)
    pos = torch.tensor([0, 1, 2, 64 * table.shape[1], -1, 5], dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 0, 1, 0, 0, 2], dtype=torch.int32, device="cuda")
    for fmt in (A.BF16, A.FP8, A.FP4):
        cache = torch.zeros(pages * kv * A.head_bytes(fmt, D), dtype=torch.uint8, device="cuda")
        dt = torch.from_numpy(table).cuda()
        ctx.kv_store(k, v, pos, seq, dt, cache, pages, fmt)
        assert ctx.device_status() == 4 and ctx.device_status() == 0
        ko = torch.empty((kv, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        vo = torch.empty((T, kv, D), dtype=torch.bfloat16, device="cuda")
        ctx.kv_load(cache, pages, fmt, pos, seq, dt, ko, vo)
        assert ctx.device_status() == 4
        assert torch.all(ko[2:] == 0) and torch.all(vo[2:] == 0)
        if fmt == A.BF16:
            assert torch.equal(vo[:2], v[:2]) and torch.equal(ko[:2].isnan(), k[:2].isnan()) and ko[1, 0, 40].isinf()
        else:
            assert torch.all(ko[0, 0, :32].isnan()) and torch.all(ko[1, 0, 32:64].isnan())
            assert not torch.any(ko[0, 0, 32:].isnan()) and not torch.any(ko[0, 1:].isnan())
    torch.cuda.synchronize()
