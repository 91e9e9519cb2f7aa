"""Host-side refusals of the rotary, K/V cache and attention calls: every bad
argument is rejected before the device is touched (no GPU needed)."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
FAKE, GOOD = P(0x1000), P(0x100000)   # never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def L():
    from dsa_sparse_attention_store_gb300 import dsaidx
    if not os.path.exists(dsaidx.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dsaidx.lib()


def _desc(**kw):
    from dsa_sparse_attention_store_gb300.dsaidx import _RopeDesc
    d = dict(theta=10000.0, rot_dim=64, max_pos=128, layout=0, scaling=0, factor=1.0, orig_max_pos=1.0, beta_slow=1.0,
             beta_fast=32.0, mscale=1.0)
    d.update(kw)
    return _RopeDesc(**d)


def test_rope_create_refuses(L):
    h = P()

    def create(ctx=FAKE, out=None, **kw):
        return L.dsa_rope_create(ctx, ctypes.byref(h) if out is None else out, ctypes.byref(_desc(**kw)))

    assert create(ctx=None) == 1
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=1026), dict(layout=2), dict(scaling=3)):
        assert create(**kw) == 2, kw
    for kw in (dict(theta=0.0), dict(theta=float("nan")), dict(max_pos=0), dict(mscale=0.0), dict(scaling=1, factor=0.0),
               dict(scaling=2, factor=2.0, beta_slow=32.0), dict(scaling=2, factor=2.0, orig_max_pos=0.0),
               dict(scaling=1, factor=float("inf"))):
        assert create(**kw) == 1, kw
    assert not h.value
    assert L.dsa_rope_destroy(None) == 1


def test_rope_apply_refuses(L):
    def call(ctx=FAKE, rope=FAKE, x=GOOD, y=GOOD, dt=0, pos=GOOD, T=1, H=1, D=64, start=0, s=(64, 64, 64, 64)):
        return L.dsa_rope_apply(ctx, rope, x, y, dt, pos, T, H, D, start, *s, 0, None)

    assert call(ctx=None) == 1 and call(rope=None) == 1
    assert call(dt=3) == 2
    for kw in (dict(T=-1), dict(H=0), dict(D=0), dict(start=-1), dict(x=None), dict(y=None), dict(pos=None),
               dict(x=P(0x100001)), dict(x=P(0x100002), dt=2), dict(pos=P(0x100002)), dict(s=(64, 64, 128, 64))):
        assert call(**kw) == 1, kw
    assert call(T=0, x=None, y=None, pos=None) == 0


def test_kv_page_bytes(L):
    assert L.dsa_kv_page_bytes(8, 128, 0) == 8 * 2 * 64 * 256
    assert L.dsa_kv_page_bytes(8, 128, 1) == 8 * 2 * 64 * 132
    assert L.dsa_kv_page_bytes(1, 64, 2) == 2 * 64 * 34
    for a in ((0, 128, 0), (1, 96, 0), (1, 128, 3)):
        assert L.dsa_kv_page_bytes(*a) == 0


def test_kv_calls_refuse(L):
    def store(ctx=FAKE, k=GOOD, v=GOOD, s=(128, 128, 128, 128), pos=GOOD, seq=GOOD, pt=GOOD, T=1, B=1, mp=1, kv=1, D=128,
              cache=GOOD, pages=1, fmt=0, rope=None, rp=None, start=0):
        return L.dsa_kv_store(ctx, k, v, *s, pos, seq, pt, T, B, mp, kv, D, cache, pages, fmt, rope, rp, start, None)

    def load(ctx=FAKE, k=GOOD, v=GOOD, s=(128, 128, 128, 128), pos=GOOD, seq=GOOD, pt=GOOD, T=1, B=1, mp=1, kv=1, D=128,
             cache=GOOD, pages=1, fmt=0):
        return L.dsa_kv_load(ctx, cache, pages, fmt, kv, D, pos, seq, pt, T, B, mp, k, v, *s, None)

    for call in (store, load):
        assert call(ctx=None) == 1
        for kw in (dict(fmt=3), dict(D=96), dict(D=256)):
            assert call(**kw) == 2, kw
        for kw in (dict(T=-1), dict(B=0), dict(mp=0), dict(kv=0), dict(pages=0), dict(k=None), dict(v=None), dict(cache=None),
                   dict(pos=None), dict(seq=None), dict(pt=None), dict(k=P(0x100008)), dict(v=P(0x100008)),
                   dict(cache=P(0x100080)), dict(s=(128, 4, 128, 128)), dict(s=(128, 128, 129, 128))):
            assert call(**kw) == 1, kw
        assert call(T=0, k=None, v=None, cache=None, pos=None, seq=None, pt=None) == 0
    assert store(start=-1) == 1 and store(rp=P(0x100001)) == 1


def _args(**kw):
    from dsa_sparse_attention_store_gb300.dsaidx import _ATTN_PACK
    d = dict(q=GOOD, q_stride_t=128, q_stride_h=128, out=GOOD, out_stride_t=128, out_stride_h=128, lse=GOOD, cache=GOOD,
             num_pages=1, fmt=0, heads=8, kv_heads=2, head_dim=128, page_table=GOOD, max_pages=1, seq_lens=GOOD, cu_q=GOOD,
             B=1, Tq=1, mask=None, mask_words=0, scale=0.1, workspace=GOOD, ws_bytes=1 << 40)
    d.update(kw)
    return _ATTN_PACK(*((v.value or 0) if isinstance(v, P) else 0 if v is None else v for v in d.values()))


def test_attention_refuses(L):
    def tree(ctx=FAKE, **kw):
        return L.dsa_tree_attn(ctx, _args(**kw), None)

    def sparse(ctx=FAKE, sel=GOOD, k=4, **kw):
        return L.dsa_sparse_attn(ctx, _args(**kw), sel, k, None)

    for call in (tree, sparse):
        assert call(ctx=None) == 1
        for kw in (dict(fmt=5), dict(head_dim=96), dict(num_pages=1 << 26), dict(Tq=1 << 29), dict(num_pages=1 << 24, kv_heads=8),
                   dict(kv_heads=1 << 17, heads=1 << 17, fmt=1)):
            assert call(**kw) == 2, kw
        for kw in (dict(Tq=-1), dict(B=0), dict(heads=0), dict(kv_heads=3), dict(kv_heads=0), dict(max_pages=0), dict(num_pages=0),
                   dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=1e-60), dict(scale=1e300),
                   dict(mask=GOOD, mask_words=0), dict(q=None), dict(out=None), dict(cache=None), dict(page_table=None),
                   dict(seq_lens=None), dict(cu_q=None), dict(workspace=None), dict(q=P(0x100008)), dict(out=P(0x100008)),
                   dict(cache=P(0x100010)), dict(workspace=P(0x100010)), dict(q_stride_t=129), dict(q_stride_h=4),
                   dict(out_stride_t=4), dict(out_stride_h=129), dict(lse=P(0x100002)), dict(mask=P(0x100002), mask_words=1)):
            assert call(**kw) == 1, kw
        assert call(Tq=0, q=None, out=None, cache=None, workspace=None, page_table=None, seq_lens=None, cu_q=None) == 0
    assert L.dsa_tree_attn(FAKE, None, None) == 1
    for kw in (dict(k=0), dict(k=65537), dict(heads=256, kv_heads=1)):
        assert sparse(**kw) == 2, kw
    assert sparse(sel=None) == 1 and sparse(sel=P(0x100001)) == 1
    assert L.dsa_attn_workspace_size(None, 128) == 0 and L.dsa_attn_workspace_size(FAKE, 96) == 0


def test_device_is_checked_before_the_handles_are_read(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU (the handles are fake)")
    h = P()
    assert L.dsa_rope_create(FAKE, ctypes.byref(h), ctypes.byref(_desc())) == 3
    assert L.dsa_rope_apply(FAKE, FAKE, GOOD, GOOD, 0, GOOD, 1, 1, 64, 0, 64, 64, 64, 64, 0, None) == 3
    assert L.dsa_kv_store(FAKE, GOOD, GOOD, 128, 128, 128, 128, GOOD, GOOD, GOOD, 1, 1, 1, 1, 128, GOOD, 1, 0, FAKE, None, 0, None) == 3
    assert L.dsa_tree_attn(FAKE, _args(), None) == 3
    assert L.dsa_sparse_attn(FAKE, _args(), GOOD, 4, None) == 3


def test_binding_refuses_what_is_not_a_cuda_tensor(L):
    import torch
    from dsa_sparse_attention_store_gb300 import dsaidx
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    for f in (lambda: dsaidx._rows(x, torch.bfloat16, x.shape, "x"),
              lambda: dsaidx._rows(None, torch.bfloat16, (1, 1, 1), "x")):
        with pytest.raises(TypeError):
            f()
