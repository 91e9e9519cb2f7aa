"""Capped rows whose visible keys all score near -cap or near cap: their weights
are the smallest and the largest, and small and large values keep their bits."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import spans as S
from tests.span_util import SpanCase
from tests.test_gpu_spans import FMTS, SIZES, ctx  # noqa: F401

pytestmark = pytest.mark.gpu


def _case(size, fmt, cap, y, power, groups=None):
    """All keys of a page's head are the same; a row's scores are y cap before the
    cap, its values 2^power times the usual ones."""
    c = SpanCase(int(cap), *SIZES[size], 128, fmt, cap=cap, groups=groups)
    kc, ks, vc, vs = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)
    if fmt == A.BF16:                           # keys of ones, whatever the format
        kc.view(np.uint16)[...] = 0x3F80
        v = vc.view(np.uint16)
        v[...] = np.where((v & 0x7F80) > 64 << 7, v.astype(np.int64) + power * 128, 0)
    else:
        kc[...], ks[...] = 0x38 if fmt == A.FP8 else 0x22, 127
        vs[...] = vs.astype(np.int64) + power
    sign = np.where(np.arange(c.Tq)[:, None, None] % 2 == 0, 1.0, 0.95)  # neighbouring rows differ
    c.q[...] = np.float32(y * cap / (c.scale * c.D)) * sign
    c.q = A.bf16_value(A.bf16_bits(c.q))
    return c


def _check(c, out, lse):
    c.check(out, lse)
    got, want = out.double().cpu().numpy(), c.reference()[0]
    to = S.tolerance(*c.reference(), c.scale, c.D, float(c.lens.max()), c.mods["cap"])[0]
    assert np.mean(np.abs(want) > to) > 0.5     # zeros would not pass
    assert np.count_nonzero(got) > 0.9 * got.size


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", ["few", "tree", "wide"])
@pytest.mark.parametrize("cap", [20.0, 30.0, 36.0, 44.0, 50.0, 57.0, 62.0, 63.0])
def test_smallest_weights_and_small_values(ctx, fmt, size, cap):  # noqa: F811
    for y in (-1.5, -8.0):
        for power in (-10, -20, -30):
            c = _case(size, fmt, cap, y, power)
            _check(c, *c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("cap", [44.0, 62.0])
def test_smallest_weights_behind_a_prefix(ctx, fmt, cap):  # noqa: F811
    c = _case("few", fmt, cap, -8.0, -30, groups=[(2, 64), (1, 0)])
    _check(c, *c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", ["few", "tree", "wide"])
@pytest.mark.parametrize("cap,power", [(20.0, 90), (30.0, 90), (44.0, 45), (50.0, 40), (62.0, 20), (63.0, 90)])
def test_largest_weights_and_large_values(ctx, fmt, size, cap, power):  # noqa: F811
    # |v| of up to 2^2.6 each (the formats' random values), 700 of them: below the stated 2^111, or 2^(127 - 1.45 cap) and more
    c = _case(size, fmt, cap, 8.0, power)
    _check(c, *c.run(ctx))
    assert ctx.device_status() == 0
