"""The tolerance of capped scores: what a sound evaluation in fp32 stays within, and
outputs that have lost their scores do not, whatever the cap."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import spans as S

LOG2E = 1.4426950408889634
FIT = np.array([0.999999463558197, -0.33330482244491577, 0.13291031122207642, -0.05136286839842796, 0.014530066400766373])


def _case(cap, gain=3.0, D=128, n=400, seed=2):
    rng = np.random.default_rng(seed)
    q = A.bf16_value(A.bf16_bits((rng.standard_normal((3, 4, D)) * gain).astype(np.float32))).astype(np.float64)
    keys, vals = (A.bf16_value(A.bf16_bits(rng.standard_normal((512, 1, D)).astype(np.float32))).astype(np.float64) for _ in range(2))
    args = (q, 1, keys, vals, np.arange(8)[None], [n], [0, 3], D ** -0.5)
    return args, S.attend(*args, cap=cap)


def _weighed(args, capped):
    """Outputs and lse with `capped` in place of the capped scores (of q.k in fp32)."""
    q, _, keys, vals, _, (n,), _, scale = args
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for t in range(3):
        L = n - 2 + t
        s = capped((q[t] @ keys[:L, 0].T).astype(np.float32)).astype(np.float64)
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        out[t] = e @ vals[:L, 0] / e.sum(-1, keepdims=True)
        lse[t] = (m + np.log(e.sum(-1, keepdims=True)))[:, 0]
    return out, lse


def _within(ref, got, args, cap):
    to, tl = S.tolerance(*ref, args[-1], args[0].shape[-1], float(args[5][0]), cap)
    return bool(np.all(np.abs(got[0] - ref[0]) <= to)), bool(np.all(np.abs(got[1] - ref[1]) <= tl))


def _difference(scale, cap):
    """cap - 2 cap / (1 + e^2y) in fp32."""
    c, k = np.float32(cap * LOG2E), np.float32(2 * LOG2E * scale / cap)

    def f(x):
        with np.errstate(over="ignore"):
            return (np.float32(-2) * c / (1 + np.exp2(x * k, dtype=np.float32)) + c) / np.float32(LOG2E)
    return f


def _polynomial(scale, cap):
    k = np.float32(scale / cap)

    def f(x):
        y = x * k
        u, p = y * y, np.full(x.shape, np.float32(FIT[4] * cap))
        for c in FIT[3::-1]:
            p = p * u + np.float32(c * cap)
        return np.where(u <= 0.390625, p * y, _difference(scale, cap)(x))
    return f


@pytest.mark.parametrize("cap", [1e3, 1e5, 1e6, 1e8, 1e12, 1e30])
def test_lost_scores_are_not_within_it(cap):
    args, ref = _case(cap)
    assert _within(ref, ref, args, cap) == (True, True)
    assert _within(ref, _weighed(args, _polynomial(args[-1], cap)), args, cap) == (True, True)
    assert _within(ref, (np.zeros_like(ref[0]), ref[1]), args, cap)[0] is False
    assert _within(ref, _weighed(args, np.zeros_like), args, cap) == (False, False)    # an average
    if cap >= 1e6:                              # the difference, which cancels
        assert _within(ref, _weighed(args, _difference(args[-1], cap)), args, cap) == (False, False)


@pytest.mark.parametrize("cap", [0.01, 1.5, 20.0, 50.0, 62.0])
def test_narrow_caps_may_take_the_difference(cap):
    for gain in (0.5, 3.0, 12.0):
        args, ref = _case(cap, gain)
        assert _within(ref, _weighed(args, _difference(args[-1], cap)), args, cap) == (True, True)


@pytest.mark.parametrize("cap", [0.0, 0.01, 20.0, 62.0, 63.0, 1e3, 1e5, 1e9])
def test_it_is_nowhere_wider_than_an_error_of_the_cap(cap):
    args, ref = _case(cap)
    _, _, wabs, qk, far, away = ref
    extra = cap * 2.0 ** -21 + far * 3 * 2.0 ** -24 + (cap + far) * 2.0 ** -23
    to, tl = A.tolerance(*ref[:4], args[-1], 128, 400.0)
    wide = to + wabs * (2.02 * extra)[..., None] + np.abs(ref[0]) * (1.01 * 2.0 ** -8), tl + 2 * extra + away * 2.0 ** -22
    got = S.tolerance(*ref, args[-1], 128, 400.0, cap)
    assert np.all(got[0] <= wide[0]) and np.all(got[1] <= wide[1])
