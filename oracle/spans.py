"""Plain 64-bit reference of the attention of spans (capped and biased scores,
first and last places, windows) and of a step's page tables, from their
definitions. A batch that shares prefixes has no reference of its own: it is the
attention of spans over page tables that name the same pages."""
from __future__ import annotations

import numpy as np

from .attention import PAGE, tolerance as plain_tolerance, visible


def seen(i, n, L, mask_row, first, last, window):
    """Places that the i-th of a sequence's n new tokens sees, of L."""
    ctx = L - n
    place = ctx + i
    see = np.zeros(L, bool)
    lo = 0 if first is None else int(first)
    hi = int(last) if last is not None else L if mask_row is not None else place + 1
    if window:
        lo = max(lo, place - window + 1)
    see[max(lo, 0):max(hi, 0)] = True
    if mask_row is not None:
        see[ctx:] &= visible(mask_row, n)
    return np.nonzero(see)[0]


def attend(q, kv_heads, keys, vals, page_table, seq_lens, cu_q, scale, mask=None, first=None, last=None, window=0, cap=0.0,
           slopes=None):
    """As attention.attend. Also returns, per row, how much the changes of the
    scores may add to a score's error: see tolerance()."""
    Tq, H, D = q.shape
    G = H // kv_heads
    out, lse = np.zeros((Tq, H, D)), np.full((Tq, H), -np.inf)
    wabs, qk, far, away = np.zeros((Tq, H, D)), np.zeros((Tq, H)), np.zeros((Tq, H)), np.zeros((Tq, H))
    for b in range(len(seq_lens)):
        n, L = int(cu_q[b + 1] - cu_q[b]), int(seq_lens[b])
        for i in range(n):
            t = int(cu_q[b]) + i
            pos = seen(i, n, L, None if mask is None else mask[t], None if first is None else first[t],
                       None if last is None else last[t], window)
            if len(pos) == 0:
                continue
            place = L - n + i
            at = page_table[b, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
            near = np.abs(pos - place).min()
            for h in range(kv_heads):
                k, v = keys[at, h], vals[at, h]
                sl = slice(h * G, (h + 1) * G)
                s = scale * (q[t, sl] @ k.T)
                if cap:
                    with np.errstate(over="ignore"):
                        s = cap * np.tanh(s / cap)
                bias = np.zeros((G, len(pos)))
                if slopes is not None:
                    bias = slopes[sl, None].astype(np.float64) * (np.abs(pos - place) - near)
                    away[t, sl] = np.abs(slopes[sl] * near)
                    s = s - bias - slopes[sl, None].astype(np.float64) * near
                m = s.max(-1, keepdims=True)
                with np.errstate(invalid="ignore"):
                    e = np.exp(s - m)
                    z = e.sum(-1, keepdims=True)
                    w = e / z
                    out[t, sl] = w @ v
                    wabs[t, sl] = w @ np.abs(v)
                    lse[t, sl] = (m + np.log(z))[:, 0]
                    qk[t, sl] = (np.abs(q[t, sl]) @ np.abs(k).T).max(-1)
                    far[t, sl] = (np.abs(bias) * (w > 1e-12)).max(-1)
    return out, lse, wabs, qk, far, away


def tolerance(out, lse, wabs, qk, far, away, scale, D, keys, cap=0.0):
    """attention.tolerance, and what the changes add to a score's error. cap:
    tanh y = 1 - 2 / (1 + 2^z) has 2^z within 2^-22 (1 + |z| 2^-2), of which at
    most half and |z| 2^z / (1 + 2^z)^2 < 0.65 of the rest arrive, and a
    reciprocal and two roundings within 2^-23 each: below cap 2^-21. An odd
    polynomial of y, for |y| up to 0.625, is within 2^-20 of its value (its fit
    2^-20.8, six roundings of 2^-24 each). Scores under a cap that needs a running
    maximum (cap log2 e > 90) are owed that: where |y| is above 0.625, cap 2^-21 <
    2^-20 cap tanh 0.625. A capped score is at most cap and at most scale sum
    |q||k|. Bias: a rounded slope, product and sum, 3 2^-24 of the bias of a key
    with weight (one below 1e-12 has none). lse takes the nearest key's bias off at
    its end.
    The results are over the sum of the rounded weights w_i (1 + e_i), |e_i| <=
    2^-8: out = sum w_i (1 + e_i) v_i / (1 + sum w_i e_i), which is off by at most
    sum w_i |e_i| |v_i| <= 2^-8 wabs, as counted there, and by |out| |sum w_i e_i|
    <= 2^-8 |out| (1 + 2^-7) besides."""
    most = np.minimum(cap, scale * qk)
    capped = cap * 2.0 ** -21 if cap * np.log2(np.e) <= 90 else np.minimum(cap * 2.0 ** -21, most * 2.0 ** -20)
    extra = capped + far * 3 * 2.0 ** -24 + (most + far) * 2.0 ** -23
    to, tl = plain_tolerance(out, lse, wabs, qk, scale, D, keys)
    return to + wabs * (2.02 * extra)[..., None] + np.abs(out) * (1.01 * 2.0 ** -8), tl + 2 * extra + away * 2.0 ** -22


def batch_plan(old, new, table, num_pages, stack, count, T, own_from=None):
    """A step's page tables and slot maps, sequence by sequence. Returns a dict
    of what the call writes; `bad` where it reports something out of range."""
    B, width = table.shape
    table, stack = table.copy(), stack.copy()
    bad = not 0 <= count <= len(stack)
    count = min(max(count, 0), len(stack))
    keep = [0] * B if own_from is None else [int(x) for x in own_from]
    ok = [o >= 0 and k >= 0 and int(o) + max(int(n), 0) <= PAGE * width for o, n, k in zip(old, new, keep)]
    bad |= not all(ok)
    pages = lambda n: -(-int(n) // PAGE)  # noqa: E731
    pool = stack[:count].tolist()
    for b in range(B):
        if ok[b] and new[b] < 0:
            pool += table[b, keep[b]:pages(old[b])].tolist()
    lens, cu = np.zeros(B, np.int32), np.zeros(B + 1, np.int64)
    seq, pos, slot = [], [], []
    for b in range(B):
        n = int(new[b]) if ok[b] and new[b] >= 0 else 0
        cu[b + 1] = cu[b] + n
        if not ok[b] or new[b] < 0:
            continue
        lens[b] = old[b] + n
        for p in range(pages(old[b]), pages(old[b] + n)):
            table[b, p] = pool.pop() if pool else -1
        for place in range(int(old[b]), int(old[b]) + n):
            page = int(table[b, place // PAGE])
            there = 0 <= page < num_pages
            bad |= not there
            seq.append(b)
            pos.append(place)
            slot.append(page * PAGE + place % PAGE if there else -1)
    bad |= len(seq) > T
    need = sum(pages(old[b] + new[b]) - pages(old[b]) for b in range(B) if ok[b] and new[b] >= 0)
    returned = sum(max(0, pages(old[b]) - keep[b]) for b in range(B) if ok[b] and new[b] < 0)
    left = count + returned - need
    bad |= left < 0 or left > len(stack)
    pad = lambda x: np.array(x[:T] + [-1] * max(0, T - len(x)), np.int32)  # noqa: E731
    for i in range(count, min(len(pool), len(stack))):
        stack[i] = pool[i]
    return dict(table=table, stack=stack, left=min(max(left, 0), len(stack)), lens=lens, cu=cu.astype(np.int32), seq=pad(seq),
                pos=pad(pos), slot=pad(slot), bad=bool(bad))
