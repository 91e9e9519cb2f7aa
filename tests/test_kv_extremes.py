"""The K/V cache at the ends of its range: what is beyond the largest scale
saturates, what is below the smallest code becomes zero, all else keeps the
format's rounding, and the attention reads the same values."""
import numpy as np
import pytest

from oracle import attention as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [A.FP8, A.FP4])
@pytest.mark.parametrize("D", [64, 128])
def test_largest_and_smallest_values(fmt, D):
    import torch
    from dsa_sparse_attention_store_gb300 import Context, kv_page_bytes
    ctx = Context(max_pos=64)
    top, most = (2.0 ** 119, 448.0) if fmt == A.FP8 else (2.0 ** 125, 6.0)
    big = np.float32(np.finfo(np.float32).max) * np.float32(0.99)       # rounds to the largest bf16
    heads = [big, np.float32(most * top), np.float32(most * top * 1.004), np.float32(1e30), np.float32(1.2e-38), np.float32(2.0 ** -133), np.float32(0)]
    rng = np.random.default_rng(fmt + D)
    x = np.zeros((len(heads), 1, D), np.float32)
    for t, a in enumerate(heads):                # a block's largest value, and others down to 2^-12 of it
        x[t, 0] = a * np.exp2(-12 * rng.random(D)) * rng.choice([-1.0, 1.0], D)
        x[t, 0, ::32] = a
    x = A.bf16_value(A.bf16_bits(x))
    T = len(heads)
    k = torch.from_numpy(x).bfloat16().cuda()
    pos, seq = torch.arange(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cache = torch.zeros(kv_page_bytes(1, D, fmt), dtype=torch.uint8, device="cuda")
    ctx.kv_store(k, k, pos, seq, table, cache, 1, fmt)
    kc, ks, vc, vs = (f[0, 0, :T] for f in A.fields(cache.cpu().numpy(), 1, 1, D, fmt))
    for t in range(T):
        codes, scales = A.quantise(x[t, 0], fmt)
        for c, s in ((kc, ks), (vc, vs)):
            assert np.array_equal(c[t], codes) and np.array_equal(s[t], scales), (t, heads[t])
    want = A.decode(kc, ks, fmt)
    assert np.isfinite(want).all() and np.abs(want[0]).max() == most * top      # saturated: the largest bf16 is above it
    ko, vo = torch.full_like(k, 3.0), torch.full_like(k, 3.0)
    ctx.kv_load(cache, 1, fmt, pos, seq, table, ko, vo)
    for got in (ko, vo):
        assert np.array_equal(got[:, 0].double().cpu().numpy(), want)
    # one key at a time, a weight of one: the value itself
    q = torch.zeros((T, 1, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(ctx.attn_workspace_size(D), dtype=torch.uint8, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    ctx.sparse_attn(q, pos.view(T, 1), cache, 1, fmt, 1, table, i32(T), i32(0, T), out, ws)
    assert np.array_equal(out[:, 0].double().cpu().numpy(), want)
    assert ctx.device_status() == 0
    ctx.close()
