"""Host-side refusals of the calls for spans, shared prefixes and a step's page
tables: every bad argument is rejected before the device is touched (no GPU
needed); and the binding refuses tensors on another GPU."""
import ctypes
import os

import pytest

from tests.test_abi_attention import FAKE, GOOD, P, _args
from tests.test_binding_devices import ATTN, _on, _Refused, ctx, i32  # noqa: F401


@pytest.fixture(scope="module")
def L():
    from dsa_sparse_attention_store_gb300 import dsaidx
    if not os.path.exists(dsaidx.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dsaidx.lib()


def _span(first=None, last=None, slopes=None, cap=0.0, window=0):
    from dsa_sparse_attention_store_gb300.dsaidx import _SPAN_PACK
    v = lambda x: (x.value or 0) if isinstance(x, P) else 0  # noqa: E731
    return _SPAN_PACK(v(first), v(last), v(slopes), cap, window)


def test_spans_refuse(L):
    def span(c=FAKE, s=None, **kw):
        return L.dsa_span_attn(c, _args(**kw), s, None)

    def shared(c=FAKE, s=None, cu=GOOD, lens=GOOD, n=1, **kw):
        return L.dsa_shared_attn(c, _args(**kw), s, cu, lens, n, None)

    for call in (span, shared):
        assert call(c=None) == 1
        for kw in (dict(fmt=5), dict(head_dim=96), dict(num_pages=1 << 26), dict(Tq=1 << 29), dict(B=(1 << 20) + 1)):
            assert call(**kw) == 2, kw
        for kw in (dict(Tq=-1), dict(B=0), dict(kv_heads=3), dict(scale=0.0), dict(q=None), dict(out=None), dict(workspace=None),
                   dict(out_stride_t=4), dict(lse=P(0x100002))):
            assert call(**kw) == 1, kw
        for kw in (dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-300), dict(cap=1e39), dict(window=-1),
                   dict(first=P(0x100002)), dict(last=P(0x100001)), dict(slopes=P(0x100002))):
            assert call(s=_span(**kw)) == 1, kw
        assert call(s=_span(slopes=GOOD), mask=GOOD, mask_words=1) == 2      # distances of drafted tokens are not those of places
        assert call(Tq=0, q=None, out=None, cache=None, workspace=None, page_table=None, seq_lens=None, cu_q=None) == 0
    assert L.dsa_span_attn(FAKE, None, None, None) == 1 and L.dsa_shared_attn(FAKE, None, None, GOOD, GOOD, 1, None) == 1
    for kw in (dict(n=0), dict(n=-1), dict(cu=None), dict(lens=None), dict(cu=P(0x100002)), dict(lens=P(0x100001))):
        assert shared(**kw) == 1, kw
    assert shared(n=(1 << 20) + 1) == 2


def test_workspace_sizes_refuse(L):
    for a in ((1, 1, 8, 2, 96), (-1, 1, 8, 2, 64), (1, 0, 8, 2, 64), (1, 1, 8, 3, 64), (1, 1, 0, 2, 64), (1 << 29, 1, 8, 2, 64)):
        assert L.dsa_span_attn_workspace_size(FAKE, *a) == 0
        assert L.dsa_shared_attn_workspace_size(FAKE, *a[:2], 1, *a[2:]) == 0
    assert L.dsa_span_attn_workspace_size(None, 1, 1, 8, 2, 64) == 0
    assert L.dsa_shared_attn_workspace_size(FAKE, 1, 1, 0, 8, 2, 64) == 0


def test_batch_plan_refuses(L):
    def arrays(**kw):
        at = {k: P(0x100000 + 0x1000 * i) for i, k in enumerate(
            ("old", "new", "own", "table", "free", "count", "left", "lens", "cu", "seq", "pos", "slot"))}
        at.update(kw)
        return at

    def call(c=FAKE, B=2, mp=3, pages=9, cap=9, T=5, **kw):
        from dsa_sparse_attention_store_gb300.dsaidx import _BATCH_PACK
        a = arrays(**kw)
        v = [(a[k].value or 0) if a[k] is not None else 0 for k in ("old", "new", "own", "count", "table", "free", "left", "lens", "cu", "seq",
                                                                    "pos", "slot")]
        return L.dsa_batch_plan(c, _BATCH_PACK(*v, B, T, mp, pages, cap), None)

    import torch
    fine = 3                                    # got as far as asking for the device, where there is none
    if not torch.cuda.is_available():
        assert call() == fine and call(own=None, slot=None) == fine and call(T=0, seq=None, pos=None, slot=None) == fine
    assert call(c=None) == 1 and L.dsa_batch_plan(FAKE, None, None) == 1
    for kw in (dict(B=0), dict(B=-1), dict(T=-1), dict(mp=0), dict(pages=0), dict(cap=-1), dict(seq=None), dict(pos=None)):
        assert call(**kw) == 1, kw
    for k in ("old", "new", "table", "free", "count", "left", "lens", "cu"):
        assert call(**{k: None}) == 1, k
    for k in arrays():
        assert call(**{k: P(0x100002 + 0x100000)}) == 1, k
    for kw in (dict(B=65537), dict(mp=1 << 25), dict(pages=1 << 25)):
        assert call(**kw) == 2, kw
    a = arrays()
    for written in ("table", "free", "left", "lens", "cu", "seq", "pos", "slot"):       # what is written overlaps nothing
        for other in a:
            if other != written:
                assert call(**{other: a[written]}) == 1, (written, other)


SPAN = dict(ATTN, first=i32(2), last=i32(2))
CALLS = {
    "span_attn": (SPAN, dict(num_pages=1, fmt=0, kv_heads=1)),
    "shared_attn": (dict(SPAN, cu_groups=i32(2), shared_lens=i32(1)), dict(num_pages=1, fmt=0, kv_heads=1)),
    "batch_plan": (dict(old_lens=i32(1), new_lens=i32(1), page_table=i32(1, 1), free_pages=i32(1), free_count=i32(1), free_left=i32(1),
                        seq_lens=i32(1), cu_q=i32(2), seq_id=i32(2), cache_pos=i32(2), slots=i32(2), own_from=i32(1)), dict(num_pages=1)),
}


@pytest.mark.parametrize("call", CALLS)
def test_tensors_elsewhere_are_refused(ctx, call):  # noqa: F811
    tensors, rest = CALLS[call]
    run = getattr(ctx, call)
    with pytest.raises(_Refused):               # all here: the library is called
        run(**{k: _on(v, False) for k, v in tensors.items()}, **rest, stream=0)
    for bad in tensors:
        with pytest.raises(ValueError, match="device"):
            run(**{k: _on(v, k == bad) for k, v in tensors.items()}, **rest, stream=0)


def test_arguments_are_packed_as_the_header_has_them(L, tmp_path):
    import shutil
    import subprocess
    from dsa_sparse_attention_store_gb300 import dsaidx
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "span.c"
    src.write_text('#include "dsaidx.h"\n'
                   f"_Static_assert(sizeof(dsa_span) == {len(_span())} && offsetof(dsa_span, slopes) == 16 && "
                   "offsetof(dsa_span, cap) == 24 && offsetof(dsa_span, window) == 32, \"dsa_span\");\n"
                   "_Static_assert(sizeof(dsa_batch_args) == 120 && offsetof(dsa_batch_args, slots) == 88 && offsetof(dsa_batch_args, B) == 96 && "
                   "offsetof(dsa_batch_args, free_cap) == 112, \"dsa_batch_args\");\n"
                   f"_Static_assert(DSA_K_ALL == {len(dsaidx.KERNEL_KINDS)}, \"kinds\");\n")
    subprocess.run([cc, "-fsyntax-only", "-I", os.path.join(root, "include"), str(src)], check=True)
    assert ctypes.sizeof(ctypes.c_void_p) == 8
