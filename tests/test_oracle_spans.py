"""The 64-bit reference of spans and of a step's page tables, by hand on small
cases and against the plain attention's reference."""
import math

import numpy as np

from oracle import attention as A
from oracle import spans as S


def _batch(seed=3, D=64):
    rng = np.random.default_rng(seed)
    keys, vals = rng.standard_normal((256, 2, D)), rng.standard_normal((256, 2, D))
    table = np.array([[2, 0], [1, 3]])
    return rng.standard_normal((5, 4, D)), keys, vals, table, np.array([70, 66]), np.array([0, 3, 5])


def test_without_changes_it_is_the_plain_attention():
    q, keys, vals, table, lens, cu = _batch()
    mask = np.array([[1], [3], [5], [1], [2]], np.uint32)
    for m in (None, mask):
        want = A.attend(q, 2, keys, vals, table, lens, cu, 0.1, mask=m)
        got = S.attend(q, 2, keys, vals, table, lens, cu, 0.1, mask=m)
        for a, b in zip(want, got):
            assert np.allclose(a, b, rtol=1e-13, atol=1e-13)
        # a cap far above every score changes nothing; a slope of 0 neither
        got = S.attend(q, 2, keys, vals, table, lens, cu, 0.1, mask=m, cap=1e9, slopes=np.zeros(4))
        assert np.allclose(got[0], want[0], atol=1e-12) and np.allclose(got[1], want[1], atol=1e-9)


def test_seen_by_hand():
    # 4 new tokens behind 6; token 1 lies at place 7
    s = lambda **kw: S.seen(1, 4, 10, kw.get("mask"), kw.get("first"), kw.get("last"), kw.get("window", 0)).tolist()  # noqa: E731
    assert s() == list(range(8))
    assert s(first=5) == [5, 6, 7] and s(first=8) == [] and s(first=-3) == list(range(8))
    assert s(last=10) == list(range(10)) and s(last=99) == list(range(10)) and s(last=3) == [0, 1, 2] and s(last=-1) == []
    assert s(window=1) == [7] and s(window=3) == [5, 6, 7] and s(window=3, last=10) == [5, 6, 7, 8, 9]
    assert s(mask=[0b1010]) == [0, 1, 2, 3, 4, 5, 7, 9] and s(mask=[0b1010], window=3) == [5, 7, 9]
    assert s(mask=[0b1010], last=9, first=4) == [4, 5, 7]


def test_cap_and_bias_by_hand():
    # two keys with scores 3 and -1, distances 1 and 0
    q = np.array([[[1.0, 0.0]]])
    keys, vals = np.zeros((64, 1, 2)), np.zeros((64, 1, 2))
    keys[0, 0, 0], keys[1, 0, 0] = 3.0, -1.0
    vals[0, 0], vals[1, 0] = [1.0, 0.0], [0.0, 1.0]
    args = (q, 1, keys, vals, np.array([[0]]), np.array([2]), np.array([0, 1]), 1.0)
    a, b = 2 * math.tanh(1.5) - 0.25, 2 * math.tanh(-0.5)
    out, lse = S.attend(*args, cap=2.0, slopes=np.array([0.25]))[:2]
    z = math.exp(a) + math.exp(b)
    assert np.allclose(out[0, 0], [math.exp(a) / z, math.exp(b) / z]) and np.allclose(lse[0, 0], math.log(z))


def test_batch_plan_by_hand():
    table = np.full((3, 4), 90, np.int32)
    table[0, :2], table[1, :2], table[2, 0] = [5, 6], [7, 8], 9
    stack = np.array([1, 2, 3, -1, -1, -1], np.int32)
    # 0 goes from 70 to 130 tokens (one page), 1 ends (keeps its first page for another), 2 has 10 + 1
    r = S.batch_plan([70, 128, 10], [60, -1, 1], table, 100, stack, 3, 70, own_from=[0, 1, 0])
    assert not r["bad"] and r["left"] == 3 and r["lens"].tolist() == [130, 0, 11] and r["cu"].tolist() == [0, 60, 60, 61]
    assert r["table"][0].tolist() == [5, 6, 8, 90] and r["stack"].tolist() == [1, 2, 3, -1, -1, -1]
    assert r["seq"].tolist() == [0] * 60 + [2] + [-1] * 9 and r["pos"][:2].tolist() == [70, 71] and r["pos"][60] == 10
    assert r["slot"][0] == 6 * 64 + 6 and r["slot"][58] == 8 * 64 and r["slot"][60] == 9 * 64 + 10 and r["slot"][61] == -1
    # nothing taken: the page that came back goes on the stack; too few pages: -1
    r = S.batch_plan([70, 128, 10], [0, -1, 0], table, 100, stack, 3, 0, own_from=[0, 1, 0])
    assert r["left"] == 4 and r["stack"].tolist() == [1, 2, 3, 8, -1, -1] and not r["bad"]
    r = S.batch_plan([0, 0, 0], [64, 128, 65], table, 100, stack, 3, 300)
    assert r["bad"] and r["left"] == 0 and r["table"][:, :2].tolist() == [[3, 6], [2, 1], [-1, -1]] and (r["slot"][192:] == -1).all()
