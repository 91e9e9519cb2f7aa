"""Reading kernel times: a program's arrays are never written past the length
it was compiled with, whatever kinds later versions add."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INDEXER_KINDS = 5      # DSA_K_COUNT as programs before the attention calls have it


@pytest.fixture(scope="module")
def L():
    from dsa_sparse_attention_store_gb300 import dsaidx
    if not os.path.exists(dsaidx.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dsaidx.lib()


def test_header_keeps_the_length(tmp_path):
    from dsa_sparse_attention_store_gb300 import dsaidx
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    src = tmp_path / "kinds.c"
    src.write_text('#include "dsaidx.h"\n'
                   f'_Static_assert(DSA_K_COUNT == {INDEXER_KINDS}, "length of dsa_profile_read");\n'
                   f'_Static_assert(DSA_K_ALL == {len(dsaidx.KERNEL_KINDS)}, "kinds of the binding");\n')
    subprocess.run([cc, "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)], check=True)


def test_read_refuses(L):
    fake = ctypes.c_void_p(0x1000)      # never dereferenced
    ms, n = (ctypes.c_float * 10)(), (ctypes.c_int32 * 10)()
    assert L.dsa_profile_read(None, ms, n) == 1 and L.dsa_profile_read(fake, None, n) == 1
    assert L.dsa_profile_read_kinds(None, ms, n, 10) == 1 and L.dsa_profile_read_kinds(fake, ms, None, 10) == 1
    assert L.dsa_profile_read_kinds(fake, ms, n, 0) == 1 and L.dsa_profile_read_kinds(fake, ms, n, -3) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("kinds", [0, 1, 5, 7, 10, 14])     # 0: the call without a length
def test_read_stays_in_its_arrays(L, kinds):
    import torch
    from dsa_sparse_attention_store_gb300 import Context, Rope, dsaidx
    ctx = Context(max_pos=64)
    rope = Rope(ctx, rot_dim=64, max_pos=16)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    ctx.profile_enable(True)
    ctx.rope_apply(x, pos, rope)
    ctx.rope_apply(x, pos, rope)
    length = kinds or INDEXER_KINDS
    ms, n = (ctypes.c_float * 20)(*[-7.0] * 20), (ctypes.c_int32 * 20)(*[-7] * 20)
    st = L.dsa_profile_read_kinds(ctx.handle, ms, n, kinds) if kinds else L.dsa_profile_read(ctx.handle, ms, n)
    assert st == 0
    assert list(ms)[length:] == [-7.0] * (20 - length) and list(n)[length:] == [-7] * (20 - length)
    at = dsaidx.KERNEL_KINDS.index("rope")
    for k in range(length):
        assert n[k] == (2 if k == at else 0) and (ms[k] > 0) == (k == at)
    again = ctx.profile_read()              # both were reset, whether asked for or not
    assert set(again) == set(dsaidx.KERNEL_KINDS) and all(v == (0.0, 0) for v in again.values())
    rope.close()
    ctx.close()
