"""Outputs whose rows share elements (an expanded tensor, strides that are too
small) are refused: the rows' threads would write them in any order."""
import ctypes
import os
import random

import pytest

P = ctypes.c_void_p
FAKE, GOOD, ELSE = P(0x1000), P(0x100000), P(0x900000)   # never dereferenced


@pytest.fixture(scope="module")
def L():
    from dsa_sparse_attention_store_gb300 import dsaidx
    if not os.path.exists(dsaidx.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dsaidx.lib()


def _meet(n0, s0, n1, s1, width):
    """By writing every row down."""
    seen = set()
    for i in range(n0):
        for j in range(n1):
            row = range(i * s0 + j * s1, i * s0 + j * s1 + width)
            if not seen.isdisjoint(row):
                return True
            seen.update(row)
    return False


def _layouts(unit, width):
    """(T, token stride, H, head stride) of every kind, strides multiples of `unit`."""
    rng = random.Random(7)
    yield from [(3, 0, 2, width), (3, 2 * width, 2, 0), (1, 0, 2, 0), (2, 0, 1, 0), (3, width, 2, width), (4, width - unit, 1, 0),
                (3, width, 2, width - unit), (3, 2 * width, 2, width), (1, 0, 1, 0), (1, 0, 4, width), (4, width, 1, 0),
                (3, width, 2, 3 * width), (3, 2 * width, 3, 3 * width), (2, 2 * width, 2, 3 * width), (3, -2 * width, 2, width)]
    for _ in range(300):
        yield (rng.randint(1, 5), unit * rng.randint(-4 * width // unit, 4 * width // unit), rng.randint(1, 5),
               unit * rng.randint(-4 * width // unit, 4 * width // unit))


def _cases(unit, width):
    """Layouts and the status to expect: refused, or past the arguments' checks to
    the device, which is not there (with one, the made-up context must not be
    looked at, so only the refused layouts are tried)."""
    import torch
    for layout in _layouts(unit, width):
        if _meet(*layout, width):
            yield layout, 1
        elif not torch.cuda.is_available():
            yield layout, 3


def test_rope_refuses_rows_that_meet(L):
    seen = set()
    for (T, st, H, sh), want in _cases(1, 6):
        assert L.dsa_rope_apply(FAKE, FAKE, GOOD, ELSE, 0, GOOD, T, H, 6, 0, 6, 6, st, sh, 0, None) == want, (T, st, H, sh)
        seen.add(want)
    assert 1 in seen


def test_kv_load_refuses_rows_that_meet(L):
    for (T, st, H, sh), want in _cases(8, 64):
        for s in ((st, sh, 64 * H, 64), (64 * H, 64, st, sh)):
            assert L.dsa_kv_load(FAKE, GOOD, 1, 0, H, 64, GOOD, GOOD, GOOD, T, 1, 1, GOOD, ELSE, *s, None) == want, (T, H, s)


def test_attention_refuses_rows_that_meet(L):
    from dsa_sparse_attention_store_gb300.dsaidx import _ATTN_PACK
    for (T, st, H, sh), want in _cases(8, 64):
        args = _ATTN_PACK(GOOD.value, 0, 0, ELSE.value, st, sh, GOOD.value, GOOD.value, 1, 0, H, 1, 64, GOOD.value, 1, GOOD.value,
                          GOOD.value, 1, T, 0, 0, 0.1, GOOD.value, 1 << 40)
        assert L.dsa_tree_attn(FAKE, args, None) == want, (T, st, H, sh)
        assert L.dsa_sparse_attn(FAKE, args, GOOD, 4, None) == want, (T, st, H, sh)


@pytest.mark.gpu
def test_binding_refuses_expanded_outputs():
    import torch
    from dsa_sparse_attention_store_gb300 import Context, Rope, dsaidx, kv_page_bytes
    ctx = Context(max_pos=64)
    rope = Rope(ctx, rot_dim=32, max_pos=16)
    new = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")    # noqa: E731
    x, pos, seq, table = new(3, 2, 64), i32(0, 1, 2), i32(0, 0, 0), i32(0).view(1, 1)
    cache = torch.zeros(kv_page_bytes(2, 64, 0), dtype=torch.uint8, device="cuda")
    ws = torch.empty(ctx.attn_workspace_size(64), dtype=torch.uint8, device="cuda")
    calls = [lambda y: ctx.rope_apply(x, pos, rope, out=y), lambda y: ctx.kv_load(cache, 1, 0, pos, seq, table, y, new(3, 2, 64)),
             lambda y: ctx.kv_load(cache, 1, 0, pos, seq, table, new(3, 2, 64), y),
             lambda y: ctx.tree_attn(x, cache, 1, 0, 2, table, i32(3), i32(0, 3), y, ws),
             lambda y: ctx.sparse_attn(x, i32(0, 1, 2).view(3, 1), cache, 1, 0, 2, table, i32(3), i32(0, 3), y, ws),
             lambda y: ctx.rope_apply(y, pos, rope)]
    for call in calls:
        for bad in (new(1, 2, 64).expand(3, -1, -1), new(3, 1, 64).expand(-1, 2, -1), new(1, 1, 64).expand(3, 2, 64)):
            with pytest.raises(dsaidx.DsaError) as e:
                call(bad)
            assert e.value.status == 1
        for good in (new(3, 2, 64), new(2, 3, 64).transpose(0, 1), new(3, 4, 64)[:, ::2], new(6, 2, 128)[::2, :, 64:], new(1, 3, 2, 64)[0]):
            call(good)
    # in place only the rotated part is written: rows may lie closer than their whole width
    flat = torch.randn(4 * 32 + 32, device="cuda").bfloat16()
    y = flat.as_strided((4, 1, 64), (32, 32, 1))
    want = flat.clone()
    for t in range(4):
        ctx.rope_apply(want[32 * t:32 * t + 32].view(1, 1, 32), i32(t), rope)
    ctx.rope_apply(y, i32(0, 1, 2, 3), rope)
    assert torch.equal(flat, want)
    assert ctx.device_status() == 0
    rope.close()
    ctx.close()
