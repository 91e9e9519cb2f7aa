"""Plain 64-bit reference of the operators that follow the indexer: rotary
positions, the K/V cache's formats, attention over the cache (tree and
selection forms). Straight from the definitions in include/dsaidx.h; no code
shared with the library."""
from __future__ import annotations

import math

import numpy as np

PAGE = 64
BF16, FP8, FP4 = 0, 1, 2


# ------------------------------------------------------------------ rotary positions

def frequencies(rot, theta=10000.0, scaling="none", factor=1.0, orig=32768.0, slow=1.0, fast=32.0):
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=np.float64)
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        g = np.clip((orig * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        return f / factor * (1.0 - g) + f * g
    return f


def rope(x, pos, rot, start, layout, freq, mscale=1.0, inverse=False):
    """x [T, H, D] float64 -> the rotated rows, float64."""
    y = np.array(x, dtype=np.float64)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * freq[None, :]
    c, s = mscale * np.cos(ang), mscale * np.sin(ang)
    if inverse:
        s = -s
    for i in range(rot // 2):
        a, b = (start + i, start + i + rot // 2) if layout == "half" else (start + 2 * i, start + 2 * i + 1)
        u, w = x[:, :, a].astype(np.float64), x[:, :, b].astype(np.float64)
        y[:, :, a] = u * c[:, None, i] - w * s[:, None, i]
        y[:, :, b] = w * c[:, None, i] + u * s[:, None, i]
    return y


# ------------------------------------------------------------------ cache formats

E4M3 = np.array([(-1.0 if c & 0x80 else 1.0) * ((c & 7) / 8.0 * 2.0 ** -6 if not (c >> 3) & 15 else
                                              (1 + (c & 7) / 8.0) * 2.0 ** (((c >> 3) & 15) - 7)) for c in range(256)])
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def code_bytes(fmt, D):
    return {BF16: 2 * D, FP8: D, FP4: D // 2}[fmt]


def scale_bytes(fmt, D):
    return 0 if fmt == BF16 else D // 32


def head_bytes(fmt, D):
    return 2 * PAGE * (code_bytes(fmt, D) + scale_bytes(fmt, D))


def bf16_bits(x):
    """Round to nearest even, as uint16 bits (NaN stays a NaN). x is float32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    r = ((b.astype(np.uint64) + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), r)


def bf16_value(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def quantise(y, fmt):
    """One row of float32 values [D] -> (codes uint8, scales uint8)."""
    D = y.shape[0]
    if fmt == BF16:
        return bf16_bits(y).view(np.uint8), np.zeros(0, np.uint8)
    most, lo, hi = (448.0, -117, 119) if fmt == FP8 else (6.0, -125, 125)
    codes, scales = np.zeros(D, np.uint8), np.zeros(D // 32, np.uint8)
    for i in range(D // 32):
        b = y[32 * i:32 * i + 32].astype(np.float64)
        if not np.all(np.isfinite(b)):
            scales[i] = 255
            continue
        amax = np.abs(b).max()
        e = lo
        while e < hi and amax > most * 2.0 ** e:
            e += 1
        scales[i] = e + 127
        table = (E4M3[:127] if fmt == FP8 else E2M1[:8])     # non-negative values, ascending
        mag = np.minimum(np.abs(b) / 2.0 ** e, most)
        up = np.minimum(np.searchsorted(table, mag, side="left"), len(table) - 1)
        dn = np.maximum(up - 1, 0)
        du, dd = table[up] - mag, mag - table[dn]
        c = np.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, dn)
        codes[32 * i:32 * i + 32] = c + np.where(np.signbit(b), 128 if fmt == FP8 else 8, 0)
    if fmt == FP4:
        return (codes[0::2] | (codes[1::2] << 4)).astype(np.uint8), scales
    return codes, scales


def decode(codes, scales, fmt):
    """codes [..., code bytes], scales [..., D/32] -> float64 [..., D]."""
    if fmt == BF16:
        return bf16_value(np.ascontiguousarray(codes).view(np.uint16)).astype(np.float64)
    if fmt == FP8:
        v = E4M3[codes]
    else:
        v = E2M1[np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def fields(cache, num_pages, kv, D, fmt):
    """Views of the byte cache: (K codes, K scales, V codes, V scales), each
    [pages, kv, 64, n]."""
    cb, sb = code_bytes(fmt, D), scale_bytes(fmt, D)
    c = cache[:num_pages * kv * head_bytes(fmt, D)].reshape(num_pages, kv, -1)
    cut = lambda at, n: c[:, :, at:at + PAGE * n].reshape(num_pages, kv, PAGE, n)  # noqa: E731
    return (cut(0, cb), cut(2 * PAGE * cb, sb), cut(PAGE * cb, cb), cut(2 * PAGE * cb + PAGE * sb, sb))


def values(cache, num_pages, kv, D, fmt):
    """The cache's keys and values, float64 [pages * 64, kv, D]."""
    kc, ks, vc, vs = fields(cache, num_pages, kv, D, fmt)
    flat = lambda x: np.ascontiguousarray(x.transpose(0, 2, 1, 3)).reshape(num_pages * PAGE, kv, D)  # noqa: E731
    return flat(decode(kc, ks, fmt)), flat(decode(vc, vs, fmt))


def random_cache(rng, num_pages, kv, D, fmt, spread=1.0):
    """A cache of random valid contents (uint8)."""
    n = num_pages * kv * head_bytes(fmt, D)
    cache = np.zeros(n, np.uint8)
    kc, ks, vc, vs = fields(cache, num_pages, kv, D, fmt)
    for codes, scales in ((kc, ks), (vc, vs)):
        assert np.shares_memory(codes, cache)
        if fmt == BF16:
            codes[...] = bf16_bits((rng.standard_normal((*codes.shape[:3], D)) * spread).astype(np.float32)).view(np.uint8)
        else:
            c = rng.integers(0, 256, codes.shape, dtype=np.uint8)
            if fmt == FP8:
                c = np.where((c & 0x7F) == 0x7F, c & 0x80, c).astype(np.uint8)   # no NaN codes: never written
                c = np.where((c & 0x7F) > 0x60, (c & 0x80) | 0x30, c).astype(np.uint8)
            codes[...] = c
            scales[...] = rng.integers(-6 if fmt == FP8 else -2, -3 if fmt == FP8 else 0, scales.shape) + 127
    return cache


# ------------------------------------------------------------------ attention

def visible(mask_row, n):
    """Truth values of the first n bits of a row of uint32 words."""
    bits = np.unpackbits(np.ascontiguousarray(mask_row, dtype=np.uint32).view(np.uint8), bitorder="little")
    out = np.zeros(n, bool)
    m = min(n, bits.shape[0])
    out[:m] = bits[:m].astype(bool)
    return out


def attend(q, kv_heads, keys, vals, page_table, seq_lens, cu_q, scale, mask=None, sel=None, slots=False):
    """q float64 [Tq, H, D]; keys/vals [slots, kv, D]. Returns out, lse and the
    two sums a tolerance is made of: per row sum w|v| [Tq, H, D] and the
    largest sum |q||k| of a visible key [Tq, H]."""
    Tq, H, D = q.shape
    G = H // kv_heads
    out, lse = np.zeros((Tq, H, D)), np.full((Tq, H), -np.inf)
    wabs, qk = np.zeros((Tq, H, D)), np.zeros((Tq, H))
    for b in range(len(seq_lens)):
        n, L = int(cu_q[b + 1] - cu_q[b]), int(seq_lens[b])
        for i in range(n):
            t = int(cu_q[b]) + i
            ctx = L - n
            if sel is None:
                pos = np.arange(ctx)
                see = visible(mask[t], n) if mask is not None else np.arange(n) <= i
                pos = np.concatenate([pos, ctx + np.nonzero(see)[0]])
            else:
                pos = sel[t][sel[t] >= 0].astype(np.int64)
                if mask is not None:
                    tree = ctx + np.nonzero(visible(mask[t], n))[0]
            slot = lambda p: page_table[b, p // PAGE].astype(np.int64) * PAGE + p % PAGE  # noqa: E731
            if sel is None:
                at = slot(pos)
            else:
                at = pos if slots else slot(pos)
                if mask is not None:
                    at = np.concatenate([at, slot(tree)])
            if len(at) == 0:
                continue
            for h in range(kv_heads):
                k, v = keys[at, h], vals[at, h]
                qq = q[t, h * G:(h + 1) * G]
                s = scale * (qq @ k.T)
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                z = e.sum(-1, keepdims=True)
                w = e / z
                sl = slice(h * G, (h + 1) * G)
                with np.errstate(invalid="ignore"):
                    out[t, sl] = w @ v
                    wabs[t, sl] = w @ np.abs(v)
                lse[t, sl] = (m + np.log(z))[:, 0]
                qk[t, sl] = (np.abs(qq) @ np.abs(k).T).max(-1)
    return out, lse, wabs, qk


def tolerance(out, lse, wabs, qk, scale, D, keys):
    """How far a result may be off, from its roundings alone. Scores: fp32 sums
    of D exact products, within (D + 1) 2^-24 of sum |q||k|, and one more
    rounding of x = s scale log2(e) - m; 2^x within 2^-22. A score's error is a
    relative error of its weight, twice (the sum moves too). Weights are
    rounded to bf16 for the product (2^-8) and so is the result (2^-8); sums
    over the keys in fp32 (2^-24 for every addition in a row's chain: 16 in a
    tile, one a tile)."""
    ds = scale * qk * (D + 1) * 2.0 ** -24 + np.where(np.isfinite(lse), np.abs(lse) + scale * qk, 0) * 2.0 ** -23 + 2.0 ** -22
    chain = (20 + keys / 64) * 2.0 ** -24
    rel = 2 * ds + 2.0 ** -8 + 2 * chain + 2.0 ** -20
    tol_out = np.abs(out) * 2.0 ** -8 + wabs * rel[..., None] * 1.01 + 1e-37
    tol_lse = ds + 2 * chain + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22 + 2.0 ** -22
    return tol_out, tol_lse
