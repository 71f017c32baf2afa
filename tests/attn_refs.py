"""Attention and its paged cache in float64 numpy and plain Python, straight from their definitions."""

import numpy as np


def attend(q, k, v, scale, window=0, sinks=0, positions=None):
    """(y, magnitude, lse, bound) of queries q [n, Hq, d] that are the last of the sequence of keys k [m, Hkv, d], or
    at `positions`.  Magnitude: the weighted mean of |v|, which a weight's rounding is proportional to; bound: of the
    relative error that rounding in fp32 gives a weight."""
    n, Hq, d = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    y, mag = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, bound = np.full((n, Hq), -np.inf), np.zeros((n, Hq, 1))
    p = (np.arange(m - n, m) if positions is None else np.asarray(positions))[:, None]
    j = np.arange(m)[None]
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    some = seen.any(1)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        with np.errstate(invalid="ignore"):
            s = np.where(seen, scale * (q[:, h] @ np.where(np.isfinite(kh), kh, 0.0).T), -np.inf)
        top = np.where(some, s.max(1, initial=-np.inf), 0.0)[:, None]
        w = np.exp(s - top)
        total = w.sum(1, keepdims=True)
        w = w / np.where(total == 0, 1, total)
        vz = np.where(np.isfinite(vh), vh, 0.0)
        y[:, h], mag[:, h] = w @ vz, w @ np.abs(vz)
        with np.errstate(divide="ignore"):
            lse[:, h] = (np.log(total) + np.where(some[:, None], top, 0.0))[:, 0]
        size = abs(scale) * np.where(seen, np.abs(q[:, h]) @ np.abs(np.where(np.isfinite(kh), kh, 0.0)).T, 0.0)
        # products exact, d additions and the scale of 2^-24 each (the tensor core may cut: 2^-23), exp2 to 2^-20, and
        # a sum over m keys, 16 a step
        bound[:, h, 0] = 2.0 * (d + 8) * 2.0 ** -24 * size.max(1, initial=0.0) + 2.0 ** -20 + m * 2.0 ** -26
    return y, mag, lse, bound


def plan(lens, table, free, count, cu, page, T, W):
    """The plan by hand: (slots, lens, table, count, refused)."""
    B = len(lens)
    lens, table, slots = list(lens), [list(r) for r in table], [-1] * T
    cut = [min(max(c, 0), T) for c in cu] if cu is not None else list(range(B + 1))
    asked, taken, refused = 0, 0, 0
    count = min(max(count, 0), len(free))  # a height past the stack is its end
    for b in range(B):
        lo, hi = cut[b], max(cut[b], cut[b + 1])
        n, new = lens[b], hi - lo
        if n < 0:
            continue
        have, want = -(-n // page), -(-(n + new) // page)
        if want > W:
            refused += 1
            continue
        need = want - have
        asked += need
        if need and asked > count:
            refused += 1
            continue
        for i in range(need):
            table[b][have + i] = free[count - 1 - (asked - need) - i]
        if need:
            taken = asked
        for t in range(lo, hi):
            p = n + t - lo
            block = table[b][p // page]
            slots[t] = block * page + p % page if 0 <= block * page + p % page < 2 ** 31 else -1
        lens[b] = n + new
    return slots, lens, table, count - taken, refused


def paged(cache, blocks, n):
    """The first n tokens [n, Hkv, d] behind these blocks of a cache [blocks, Hkv, page, d]."""
    return np.concatenate([cache[i].transpose(1, 0, 2) for i in blocks] or [np.zeros((0,) + cache.shape[1:4:2])])[:n]
