"""The 64-bit reference of rotary positions, cache formats and attention,
checked by hand on small cases."""
import math

import numpy as np

from oracle import attention as A


def test_rope_by_hand():
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1, 2, 3, 4]
    f = np.array([math.pi / 2, 0.0])
    half = A.rope(x, [1], 4, 0, "half", f)[0, 0]
    assert np.allclose(half, [-3, 2, 1, 4])
    inter = A.rope(x, [1], 4, 0, "interleaved", f)[0, 0]
    assert np.allclose(inter, [-2, 1, 3, 4])
    assert np.allclose(A.rope(half[None, None], [1], 4, 0, "half", f, inverse=True), x)
    assert np.array_equal(A.rope(x, [0], 2, 2, "half", f[:1])[0, 0], x[0, 0])


def test_scaled_frequencies():
    f = A.frequencies(128)
    assert f[0] == 1.0 and abs(f[32] - 0.01) < 1e-15
    assert np.allclose(A.frequencies(128, scaling="linear", factor=4.0), f / 4)
    g = A.frequencies(128, scaling="by_parts", factor=4.0, orig=4096.0, slow=1.0, fast=32.0)
    turns = 4096 * f / (2 * math.pi)
    assert np.array_equal(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert np.all(g[mid] < f[mid]) and np.all(g[mid] > f[mid] / 4)


def test_formats_by_hand():
    y = np.zeros(32, np.float32)
    c, s = A.quantise(y, A.FP8)
    assert s[0] == 10 and not c.any()
    y[0], y[1], y[2] = 448.0, -448.0, 17.0          # 17 lies between 16 and 18: the even code
    c, s = A.quantise(y, A.FP8)
    assert s[0] == 127 and c[0] == 0x7E and c[1] == 0xFE and A.E4M3[c[2]] == 16.0
    y[0] = 449.0                                    # one step above: the next power of two, no saturation
    c, s = A.quantise(y, A.FP8)
    assert s[0] == 128 and A.E4M3[c[0]] == 224.0
    y[:4] = [6.0, 0.25, 0.75, -5.0]
    c, s = A.quantise(y, A.FP4)
    assert s[0] == 127
    assert np.array_equal(A.decode(c, s, A.FP4)[:4], [6.0, 0.0, 1.0, -4.0])
    y[5] = np.nan
    c, s = A.quantise(y, A.FP4)
    assert s[0] == 255 and np.all(np.isnan(A.decode(c, s, A.FP4)))


def test_quantised_values_are_bf16_numbers_and_near():
    rng = np.random.default_rng(0)
    for fmt, step in ((A.FP8, 2.0 ** -4), (A.FP4, 2.0 ** -2)):
        for gain in (1e-30, 1.0, 1e30):
            y = (rng.standard_normal(128) * gain).astype(np.float32)
            c, s = A.quantise(y, fmt)
            v = A.decode(c, s, fmt)
            assert np.array_equal(A.bf16_value(A.bf16_bits(v.astype(np.float32))), v.astype(np.float32))
            block = np.abs(y.reshape(-1, 32)).max(1).repeat(32)
            assert np.all(np.abs(v - y) <= np.maximum(np.abs(y) * step, block * (2.0 ** -10 / 224 if fmt == A.FP8 else 0.25 / 3)))


def test_attention_by_hand():
    keys = np.zeros((64, 1, 2))
    vals = np.zeros((64, 1, 2))
    keys[:4, 0] = [[1, 0], [0, 1], [5, 5], [9, 9]]
    vals[:4, 0] = [[1, 2], [3, 4], [5, 6], [7, 8]]
    q = np.array([[[1.0, 0.0], [0.0, 0.0]], [[0.0, 2.0], [1.0, 1.0]]])
    table = np.zeros((1, 1), np.int32)
    out, lse, _, _ = A.attend(q, 1, keys, vals, table, [4], [0, 2], 1.0, mask=np.array([[0], [0b11]], np.uint32))
    w = np.exp([1.0, 0.0])
    assert np.allclose(out[0, 0], (w[:, None] * vals[:2, 0]).sum(0) / w.sum())
    assert np.allclose(out[0, 1], [2, 3]) and np.isclose(lse[0, 1], math.log(2))
    assert np.isclose(lse[1, 0], np.log(np.exp([0.0, 2.0, 10.0, 18.0]).sum()))
    chain = A.attend(q, 1, keys, vals, table, [4], [0, 2], 1.0)
    assert np.isclose(chain[1][0, 1], math.log(3)) and np.allclose(chain[0][1], out[1])
    picked = A.attend(q, 1, keys, vals, table, [4], [0, 2], 1.0, sel=np.array([[1, -1], [-1, -1]], np.int32))
    assert np.allclose(picked[0][0], vals[1, 0]) and np.all(picked[0][1] == 0) and np.all(np.isneginf(picked[1][1]))
