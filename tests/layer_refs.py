"""The operators around the recurrence in float64 numpy, straight from their formulas, token by token.

Each returns, next to the values, the same sums taken over magnitudes: the scale that a sum's rounding
errors are proportional to, whatever cancels in the sum itself."""

import numpy as np


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def bounds(B, T, cu):
    return [(b * T, (b + 1) * T) for b in range(B)] if cu is None else [(int(cu[b]), int(cu[b + 1])) for b in range(B)]


def conv(x, w, bias, seqs, init, act=True):
    """(y, magnitude, final state) of the causal convolution."""
    T, C = x.shape
    K = w.shape[1]
    y, mag = np.zeros((T, C)), np.zeros((T, C))
    fin = np.zeros((len(seqs), K - 1, C))
    for b, (lo, hi) in enumerate(seqs):
        head = init[b] if init is not None else np.zeros((K - 1, C))
        seen = np.concatenate([head, x[lo:hi]])
        for t in range(hi - lo):
            y[lo + t] = (seen[t:t + K] * w.T).sum(0)
            mag[lo + t] = np.abs(seen[t:t + K] * w.T).sum(0)
        fin[b] = seen[hi - lo:]
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    # silu's slope is below 1.1 in magnitude, and silu(y) is what is rounded last
    return (silu(y) if act else y), mag, fin


def scan(x, dt, A, Bm, Cm, D, z, dt_bias, seqs, init, softplus=True):
    """(y, magnitude, final state, its magnitude) of the selective scan."""
    T, Hv, dv = x.shape
    Hk, dk = Bm.shape[1:]
    hk = np.arange(Hv) // (Hv // Hk)
    s = dt + (dt_bias if dt_bias is not None else 0.0)
    if softplus:
        s = np.logaddexp(0.0, s)
    y, mag = np.zeros((T, Hv, dv)), np.zeros((T, Hv, dv))
    fin, fmag = np.zeros((len(seqs), Hv, dv, dk)), np.zeros((len(seqs), Hv, dv, dk))
    for b, (lo, hi) in enumerate(seqs):
        S = init[b].copy() if init is not None else np.zeros((Hv, dv, dk))
        M = np.abs(S)
        for t in range(lo, hi):
            decay = np.exp(s[t] * A)[:, None, None]
            put = (s[t][:, None] * x[t])[:, :, None] * Bm[t][hk][:, None, :]
            S, M = decay * S + put, decay * M + np.abs(put)
            y[t] = np.einsum("hpn,hn->hp", S, Cm[t][hk])
            mag[t] = np.einsum("hpn,hn->hp", M, np.abs(Cm[t][hk]))
        fin[b], fmag[b] = S, M
    if D is not None:
        y, mag = y + D[:, None] * x, mag + np.abs(D[:, None] * x)
    if z is not None:
        y, mag = y * silu(z), mag * np.abs(silu(z))
    return y, mag, fin, fmag


def norm(x, residual, w, eps):
    r = x + residual if residual is not None else x
    return r, w * r / np.sqrt((r * r).mean(1, keepdims=True) + eps)


def scales(y, group):
    """max |y| over each group of columns (0: a row), floored at 2^-96, over 448."""
    g = group or y.shape[1]
    parts = [np.abs(y[:, i:i + g]).max(1) for i in range(0, y.shape[1], g)]
    return np.maximum(np.stack(parts, 1), 2.0 ** -96) / 448.0
