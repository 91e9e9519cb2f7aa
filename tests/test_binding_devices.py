"""A tensor on another GPU than the current one is refused by the binding of
the attention calls, whichever argument it is; the kernels would read an
address that is not theirs. Stand-ins for CUDA tensors: no GPU needed."""
import pytest
import torch

from dsa_sparse_attention_store_gb300 import dsaidx

HERE, THERE = 0, 1


class _On(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    at = HERE
    is_cuda = True

    def get_device(self):
        return self.at


class _Elsewhere(_On):
    at = THERE


class _Refused(Exception):
    pass


class _Lib:
    """The library, reached only when every argument has passed."""

    def __getattr__(self, name):
        if name == "dsa_kv_page_bytes":
            return lambda kv, D, fmt: 1
        def call(*args):
            raise _Refused(name)
        return call


class _Rope:
    def _open(self):
        return 1


def _on(t, there):
    return t.as_subclass(_Elsewhere if there else _On)


bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)      # noqa: E731
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)        # noqa: E731
u8 = lambda n: torch.zeros(n, dtype=torch.uint8)          # noqa: E731

ATTN = dict(q=bf(2, 4, 64), cache=u8(64), page_table=i32(1, 1), seq_lens=i32(1), cu_q=i32(2), out=bf(2, 4, 64), workspace=u8(8),
            mask=i32(2, 1), lse=torch.zeros(2, 4))
CALLS = {
    "rope_apply": (dict(x=bf(2, 4, 64), pos=i32(2), out=bf(2, 4, 64)), dict(rope=_Rope())),
    "kv_store": (dict(k=bf(2, 1, 64), v=bf(2, 1, 64), cache_pos=i32(2), seq_id=i32(2), page_table=i32(1, 1), cache=u8(64), rope_pos=i32(2)),
                 dict(num_pages=1, fmt=0, rope=_Rope())),
    "kv_load": (dict(cache=u8(64), cache_pos=i32(2), seq_id=i32(2), page_table=i32(1, 1), k=bf(2, 1, 64), v=bf(2, 1, 64)),
                dict(num_pages=1, fmt=0)),
    "tree_attn": (ATTN, dict(num_pages=1, fmt=0, kv_heads=1)),
    "sparse_attn": (dict(ATTN, sel=i32(2, 3)), dict(num_pages=1, fmt=0, kv_heads=1)),
}


@pytest.fixture()
def ctx(monkeypatch):
    monkeypatch.setattr(dsaidx, "_current_device", lambda: HERE, raising=False)
    monkeypatch.setattr(dsaidx, "_lib", _Lib())
    monkeypatch.setattr(dsaidx, "_KV_PAGE_BYTES", {})
    c = object.__new__(dsaidx.Context)
    c._h = None
    return c


@pytest.mark.parametrize("call", CALLS)
def test_tensors_elsewhere_are_refused(ctx, call):
    tensors, rest = CALLS[call]
    run = getattr(ctx, call)
    with pytest.raises(_Refused):                 # all here: the library is called
        run(**{k: _on(v, False) for k, v in tensors.items()}, **rest, stream=0)
    for bad in tensors:
        with pytest.raises(ValueError, match="device"):
            run(**{k: _on(v, k == bad) for k, v in tensors.items()}, **rest, stream=0)
