"""Float64 definitions of the gated linear recurrence and of values held in 8 and 4
bits.  Plain numpy loops from the formulas in include/gdn.h; the recurrence's
functions also return, for each result, the magnitude that an fp32 evaluation's
rounding errors are proportional to.
"""
from __future__ import annotations

import numpy as np

from .layer import f64, kept_column, ranges, start_column

GROUP = 32


def _rows(x, D):
    return None if x is None else f64(x).reshape(-1, D)


def scan(x, g, beta=None, initial_state=None, cu_seqlens=None):
    """Returns (y, final state, magnitude of y, of the final state).  A step's error is at
    most the one before times e^g, and roundings of e^g h, of beta x and of their sum."""
    B, T, D = x.shape
    xs, gs, bs, init = _rows(x, D), _rows(g, D), _rows(beta, D), f64(initial_state)
    seqs = ranges(B, T, cu_seqlens)
    y, mag = np.zeros((B * T, D)), np.zeros((B * T, D))
    final, mfinal = np.zeros((len(seqs), D)), np.zeros((len(seqs), D))
    for n, (t0, t1) in enumerate(seqs):
        h, m = (np.zeros(D) if init is None else init[n].copy()), np.zeros(D)
        for t in range(t0, t1):
            a, u = np.exp(gs[t]), xs[t] if bs is None else bs[t] * xs[t]
            m = a * (m + np.abs(h)) + np.abs(u)
            h = a * h + u
            m = m + np.abs(h)
            y[t], mag[t] = h, m
        final[n], mfinal[n] = h, m
    return y.reshape(B, T, D), final, mag.reshape(B, T, D), mfinal


def scan_steps(x, g, pool, indices, beta=None, num_accepted=None, cu_seqlens=None):
    """Returns (y, pool after, magnitude of y, of the pool)."""
    B, T, D = x.shape
    pool, idx = f64(pool), f64(indices)
    idx = idx.reshape(idx.shape[0], -1)
    cols, P, seqs = idx.shape[1], pool.shape[0], ranges(B, T, cu_seqlens)
    start = [int(idx[n, start_column(num_accepted, n, cols)]) for n in range(len(seqs))]
    live = [0 <= s < P for s in start]
    init = np.stack([pool[s] if ok else np.zeros(D) for s, ok in zip(start, live)])
    y, _, mag, _ = scan(x, g, beta, init, cu_seqlens)
    y, mag, after, mafter = y.reshape(-1, D), mag.reshape(-1, D), pool.copy(), np.zeros_like(pool)
    for n, (t0, t1) in enumerate(seqs):
        if not live[n]:
            y[t0:t1] = 0
            continue
        for i in range(t1 - t0):
            c = kept_column(i, t1 - t0, cols)
            if c is not None and 0 <= idx[n, c] < P:
                after[int(idx[n, c])], mafter[int(idx[n, c])] = y[t0 + i], mag[t0 + i]
    return y.reshape(B, T, D), after, mag.reshape(B, T, D), mafter


def scan_bwd(x, g, y, dy, beta=None, dht=None, initial_state=None, cu_seqlens=None):
    """Returns {name: (gradient, magnitude)} for dx, dg, dbeta (with beta) and dinitial;
    the state before a token is the given y of the token before, or the initial state."""
    B, T, D = dy.shape
    xs, gs, bs, ys, dys = (_rows(t, D) for t in (x, g, beta, y, dy))
    init, dend = f64(initial_state), f64(dht)
    seqs = ranges(B, T, cu_seqlens)
    out = {k: (np.zeros((B * T, D)), np.zeros((B * T, D))) for k in ("dx", "dg", "dbeta")}
    d0, m0 = np.zeros((len(seqs), D)), np.zeros((len(seqs), D))
    for n, (t0, t1) in enumerate(seqs):
        carry = np.zeros(D) if dend is None else dend[n].copy()
        m = np.abs(carry)
        for t in range(t1 - 1, t0 - 1, -1):
            dh = dys[t] + carry
            m = m + np.abs(dys[t]) + np.abs(dh)
            a = np.exp(gs[t])
            before = ys[t - 1] if t > t0 else np.zeros(D) if init is None else init[n]
            b = np.ones(D) if bs is None else bs[t]
            out["dx"][0][t], out["dx"][1][t] = b * dh, np.abs(b) * m
            out["dg"][0][t], out["dg"][1][t] = a * before * dh, a * np.abs(before) * m
            if bs is not None:
                out["dbeta"][0][t], out["dbeta"][1][t] = xs[t] * dh, np.abs(xs[t]) * m
            carry, m = a * dh, a * m
        d0[n], m0[n] = carry, m
    out = {k: (v.reshape(B, T, D), w.reshape(B, T, D)) for k, (v, w) in out.items()}
    if bs is None:
        del out["dbeta"]
    out["dinitial"] = (d0, m0)
    return out


def hold(v, bits=8):
    """v [..., D] -> (codes int64 [..., D], scales [..., groups]): see gdn_held."""
    v = f64(v)
    top, D = (127, 7)[bits == 4], v.shape[-1]
    rows = v.reshape(-1, D)
    codes, scales = np.zeros(rows.shape, dtype=np.int64), np.zeros((rows.shape[0], -(-D // GROUP)))
    for k in range(scales.shape[1]):
        part = rows[:, k * GROUP:(k + 1) * GROUP]
        bad = ~np.isfinite(part).all(-1)
        high = np.where(bad, 0.0, np.abs(np.where(np.isfinite(part), part, 0.0)).max(-1))
        m, e = np.frexp(high / top)              # high / top is exact where it has few bits: ties included
        s = np.ldexp(np.ceil(m * 256), e - 8)    # a bf16 number has 8 significant bits
        s[high < 2.0 ** -100] = 0.0
        q = np.where(s[:, None] > 0, np.where(np.isfinite(part), part, 0.0) / np.where(s > 0, s, 1.0)[:, None], 0.0)
        codes[:, k * GROUP:(k + 1) * GROUP] = np.where(bad[:, None], 0, np.rint(q))
        scales[:, k] = np.where(bad, np.nan, s)
    return codes.reshape(v.shape), scales.reshape(*v.shape[:-1], -1)


def restore(codes, scales):
    """The values that codes [..., D] and scales [..., groups] stand for."""
    codes, scales = f64(codes), f64(scales)
    return codes * np.repeat(scales, GROUP, -1)[..., :codes.shape[-1]]


def pack4(codes):
    """Codes of 4 bits [..., D] as bytes [..., (D+1)//2], element 2i in the low half."""
    codes = np.asarray(codes)
    if codes.shape[-1] % 2:
        codes = np.concatenate([codes, np.zeros((*codes.shape[:-1], 1), dtype=codes.dtype)], -1)
    return ((codes[..., 0::2] & 15) | (codes[..., 1::2] & 15) << 4).astype(np.uint8)
