"""Caps far above the scores: the capped score of a key is then nearly its
score, and has to be as exact, whatever the cap."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import spans as S
from tests.span_util import SpanCase
from tests.test_gpu_spans import FMTS, SIZES, ctx  # noqa: F401

pytestmark = pytest.mark.gpu


def _check(c, out, lse, ref, rows=None):
    """Against `ref` within the tolerance of scores that are not capped, and 2^-20
    of the largest one: tanh y by an odd polynomial of y is within 2^-20.8 of
    itself (its least coefficient, 1 - 2^-20.8, decides for small y) and six fp32
    roundings, 2^-21.4 of which are 2^-24 each; the subtraction of the exponent
    rounds once more (2^-23)."""
    to, tl = S.tolerance(*ref, c.scale, c.D, float(c.lens.max()))
    extra = np.minimum(c.mods["cap"], c.scale * ref[3]) * (2.0 ** -20 + 2.0 ** -23)
    to, tl = to + ref[2] * (2.02 * extra)[..., None], tl + 2 * extra
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = slice(None) if rows is None else rows
    assert np.all(np.abs(gl - ref[1])[rows] <= tl[rows]), float((np.abs(gl - ref[1]) / tl)[rows].max())
    assert np.all(np.abs(got - ref[0])[rows] <= to[rows]), float((np.abs(got - ref[0]) / to)[rows].max())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", ["few", "tree", "wide"])
@pytest.mark.parametrize("cap", [64.0, 3e3, 1e4, 1e6, 1e8, 1e12, 1e30, 2e36])
def test_scores_keep_their_bits_under_any_cap(ctx, fmt, D, size, cap):  # noqa: F811
    c = SpanCase(3, *SIZES[size], D, fmt, cap=cap)
    out, lse = c.run(ctx)
    _check(c, out, lse, c.reference())
    if cap >= 1e8:                              # s - cap tanh(s / cap) < s^3 / (3 cap^2): as if there were none
        c.mods["cap"] = 0.0
        ref = c.reference()
        c.mods["cap"] = cap
        _check(c, out, lse, ref)
    assert ctx.device_status() == 0


@pytest.mark.parametrize("cap", [1e5, 1e8])
@pytest.mark.parametrize("slopes", [None, True])
@pytest.mark.parametrize("size", SIZES)
def test_scores_beside_ones_at_the_cap(ctx, cap, slopes, size):  # noqa: F811
    # ten keys whose scores lie around -cap, and have no weight, in the tile of others with usual scores
    ctx_lens, nds, kv, G = SIZES[size]
    c = SpanCase(4, [n + 70 for n in ctx_lens], nds, kv, G, 128, A.BF16, cap=cap, slopes=slopes)
    c.q[...] = np.abs(c.q)                      # rows that a vector of negative numbers is far from
    kc = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)[0].view(np.uint16)
    far = A.bf16_bits(np.float32(-cap / (c.scale * c.D)))
    for b in range(c.B):
        kc[c.table[b, 0], :, :10] = far
    c.mods["first"] = np.full(c.Tq, 10, np.int32)
    ref = c.reference()                         # without those keys: e^-cap is no weight
    c.mods["first"] = None
    z = c.reference()[1]
    assert np.allclose(z, ref[1], rtol=0, atol=1e-9)
    out, lse = c.run(ctx)
    _check(c, out, lse, ref)
    assert ctx.device_status() == 0


@pytest.mark.parametrize("slopes", [None, True])
def test_keys_at_the_largest_caps(ctx, slopes):  # noqa: F811
    # ten equal keys at 0.7 cap and more, beside others with usual scores: they share the weight
    cap = 2.2e38
    c = SpanCase(5, [300], [3], 1, 4, 128, A.BF16, cap=cap, slopes=None if slopes is None else np.zeros(4))
    c.scale = 1.0
    c.q[...] = np.abs(c.q)
    kc, _, vc, _ = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)
    page = c.table[0, 1]
    far = A.bf16_bits(np.array([cap * 0.3 / c.D], np.float32))
    kc.view(np.uint16)[page, 0, 20:30] = far
    v = A.bf16_value(vc.view(np.uint16)[page, 0, 20:30]).astype(np.float64)
    out, lse = c.run(ctx)
    got = out.double().cpu().numpy()
    # equal weights, rounded alike; sums of ten and the result's rounding
    assert np.all(np.abs(got - v.mean(0)) <= 2.0 ** -8 * 1.01 * np.abs(v.mean(0)) + 2.0 ** -20 * np.abs(v).mean(0))
    y = c.q.astype(np.float64).sum(-1) * float(A.bf16_value(far)[0]) / cap
    assert np.allclose(lse.double().cpu().numpy(), cap * np.tanh(y), rtol=2.0 ** -17, atol=0)
    assert ctx.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("groups", [None, [(2, 256), (1, 0)]])
@pytest.mark.parametrize("how", ["tree", "bias", "window"])
def test_wide_caps_with_masks_biases_and_prefixes(ctx, fmt, groups, how):  # noqa: F811
    for cap in (70.0, 1e6):
        c = SpanCase(6, [400, 300, 90], [3, 40, 9], 2, 4, 128, fmt, groups=groups, masked=how == "tree", cap=cap,
                     slopes=True if how == "bias" else None, window=150 if how == "window" else 0)
        c.check(*c.run(ctx))
    assert ctx.device_status() == 0


@pytest.mark.parametrize("groups", [None, [(2, 64)]])
def test_hidden_values_under_wide_caps(ctx, groups):  # noqa: F811
    # keys and values that are not finite where no row sees them, in tiles that rows see in part
    c = SpanCase(7, [200, 150], [4, 40], 2, 4, 64, A.BF16, groups=groups, cap=1e5)
    c.mods["first"] = np.full(c.Tq, 40, np.int32)
    ref = c.reference()
    kc, _, vc, _ = A.fields(c.cache, c.pages, c.kv, c.D, c.fmt)
    for bits, codes in ((0x7F80, kc), (0x7FC0, vc)):
        for b in range(c.B):
            codes.view(np.uint16)[c.table[b, 0], :, :40] = bits
    out, lse = c.run(ctx)
    c.check(out, lse, ref=ref)
    assert ctx.device_status() == 0
