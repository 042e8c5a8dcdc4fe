"""Float64 definitions of the operators around the delta rule: the recurrent
steps over several tokens in a slot pool, the short causal convolution and the
RMS norms, with their gradients.  Plain numpy loops from the formulas in
include/gdn.h; each function also returns, where its result is computed, the
magnitude that an fp32 evaluation's rounding errors are proportional to.
"""
from __future__ import annotations

import numpy as np


def f64(x):
    """A tensor or array as a float64 (integers: int64) numpy array."""
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().cpu()
        x = x.double() if x.is_floating_point() else x.long()
        return x.numpy()
    return np.asarray(x, dtype=np.float64)


def ranges(B, T, cu_seqlens):
    if cu_seqlens is None:
        return [(n * T, n * T + T) for n in range(B)]
    cu = [int(c) for c in cu_seqlens]
    return list(zip(cu[:-1], cu[1:]))


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def start_column(num_accepted, n, cols):
    return 0 if num_accepted is None else min(max(int(num_accepted[n]), 1), cols) - 1


def kept_column(i, length, cols):
    """The column that takes the state after token i of `length`, or None."""
    if i < cols - 1:
        return i
    return cols - 1 if i == length - 1 else None


# ---------------------------------------------------------------------------
# Recurrent steps
# ---------------------------------------------------------------------------
def steps(q, k, v, g, beta, pool, indices, num_accepted=None, cu_seqlens=None, scale=None, use_l2norm=False):
    """Returns (out, pool after, bound): bound[n, j] = sum over the sequence's
    tokens of ||S||_F (|k|^2 + 1) + ||u||, S before and after the token."""
    q, k, v, g, beta, pool = (f64(x) for x in (q, k, v, g, beta, pool))
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    idx = f64(indices)
    idx = idx.reshape(idx.shape[0], -1)
    cols, P = idx.shape[1], pool.shape[0]
    q, k = q.reshape(-1, H, K), k.reshape(-1, H, K)
    v, g, beta = v.reshape(-1, HV, V), g.reshape(-1, HV), beta.reshape(-1, HV)
    if use_l2norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) for x in (q, k))
    scale = K ** -0.5 if scale is None else scale
    out, after, seqs = np.zeros_like(v), pool.copy(), ranges(B, T, cu_seqlens)
    bound = np.zeros((len(seqs), HV))
    for n, (t0, t1) in enumerate(seqs):
        slot = int(idx[n, start_column(num_accepted, n, cols)]) if t1 > t0 else -1
        if not 0 <= slot < P:
            continue
        for j in range(HV):
            S, jk = pool[slot, j].copy(), j // (HV // H)
            for t in range(t0, t1):
                kt = k[t, jk]
                before = np.linalg.norm(S)
                S = np.exp(g[t, j]) * S
                u = beta[t, j] * (v[t, j] - S.T @ kt)
                S = S + np.outer(kt, u)
                out[t, j] = scale * (S.T @ q[t, jk])
                bound[n, j] += max(before, np.linalg.norm(S)) * (kt @ kt + 1) + np.linalg.norm(u) * (1 + abs(g[t, j]))
                c = kept_column(t - t0, t1 - t0, cols)
                if c is not None and 0 <= idx[n, c] < P:
                    after[int(idx[n, c]), j] = S
    return out.reshape(B, T, HV, V), after, bound


# ---------------------------------------------------------------------------
# Short convolution
# ---------------------------------------------------------------------------
def _lines(x, W, cu_seqlens, initial):
    """Per sequence: (first token, one past the last, its inputs [W-1+len, D] with the history in front)."""
    B, T, D = x.shape
    flat = x.reshape(-1, D)
    for n, (t0, t1) in enumerate(ranges(B, T, cu_seqlens)):
        hist = np.zeros((W - 1, D)) if initial is None else initial[n].T
        yield n, t0, t1, np.concatenate([hist, flat[t0:t1]])


def conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, silu=True):
    """Returns (y, final_state, magnitude of y)."""
    x, w, b, init = f64(x), f64(weight), f64(bias), f64(initial_state)
    D, W = w.shape
    y, mag = np.zeros_like(x).reshape(-1, D), np.zeros_like(x).reshape(-1, D)
    final = np.zeros((len(ranges(x.shape[0], x.shape[1], cu_seqlens)), D, W - 1))
    for n, t0, t1, line in _lines(x, W, cu_seqlens, init):
        for t in range(t0, t1):
            rows = line[t - t0:t - t0 + W]
            pre = (rows * w.T).sum(0) + (0 if b is None else b)
            size = (np.abs(rows) * np.abs(w.T)).sum(0) + (0 if b is None else np.abs(b))
            y[t] = pre * sigmoid(pre) if silu else pre
            mag[t] = 1.1 * size + np.abs(y[t]) * (1 + np.abs(pre))
        final[n] = line[t1 - t0:].T
    return y.reshape(x.shape), final, mag.reshape(x.shape)


def conv_update(x, weight, pool, indices, bias=None, num_accepted=None, cu_seqlens=None, silu=True):
    """Returns (y, pool after, magnitude of y)."""
    x, pool, idx = f64(x), f64(pool), f64(indices)
    idx = idx.reshape(idx.shape[0], -1)
    cols, P, W = idx.shape[1], pool.shape[0], f64(weight).shape[1]
    seqs = ranges(x.shape[0], x.shape[1], cu_seqlens)
    start = [int(idx[n, start_column(num_accepted, n, cols)]) for n in range(len(seqs))]
    live = [0 <= s < P for s in start]
    init = np.stack([pool[s] if ok else np.zeros_like(pool[0]) for s, ok in zip(start, live)])
    y, _, mag = conv(x, weight, bias, init, cu_seqlens, silu)
    after, flat = pool.copy(), y.reshape(-1, x.shape[-1])
    for n, t0, t1, line in _lines(x, W, cu_seqlens, init):
        if not live[n]:
            flat[t0:t1] = 0
            continue
        for i in range(t1 - t0):
            c = kept_column(i, t1 - t0, cols)
            if c is not None and 0 <= idx[n, c] < P:
                after[int(idx[n, c])] = line[i + 1:i + W].T
    return flat.reshape(x.shape), after, mag


def conv_bwd(x, weight, dy, bias=None, initial_state=None, cu_seqlens=None, silu=True):
    """Returns {name: (gradient, magnitude)} for dx, dweight, dbias, dinitial."""
    x, w, b, init, dy = f64(x), f64(weight), f64(bias), f64(initial_state), f64(dy)
    D, W = w.shape
    dyf = dy.reshape(-1, D)
    nseq = len(ranges(x.shape[0], x.shape[1], cu_seqlens))
    g = {"dx": np.zeros_like(dyf), "dweight": np.zeros((D, W)), "dbias": np.zeros(D), "dinitial": np.zeros((nseq, D, W - 1))}
    m = {name: np.zeros_like(a) for name, a in g.items()}
    for n, t0, t1, line in _lines(x, W, cu_seqlens, init):
        dline, mline = np.zeros_like(line), np.zeros_like(line)
        for t in range(t0, t1):
            rows = line[t - t0:t - t0 + W]
            pre = (rows * w.T).sum(0) + (0 if b is None else b)
            size = (np.abs(rows) * np.abs(w.T)).sum(0) + (0 if b is None else np.abs(b))
            s = sigmoid(pre)
            dpre = dyf[t] * (s * (1 + pre * (1 - s)) if silu else 1.0)
            mpre = 1.2 * np.abs(dyf[t]) * (1 + size + np.abs(pre)) * (1 + np.abs(pre))
            for j in range(W):
                dline[t - t0 + j] += w[:, j] * dpre
                mline[t - t0 + j] += np.abs(w[:, j]) * mpre
                g["dweight"][:, j] += dpre * rows[j]
                m["dweight"][:, j] += mpre * np.abs(rows[j])
            g["dbias"] += dpre
            m["dbias"] += mpre
        g["dinitial"][n], g["dx"][t0:t1] = dline[:W - 1].T, dline[W - 1:]
        m["dinitial"][n], m["dx"][t0:t1] = mline[:W - 1].T, mline[W - 1:]
    g["dx"], m["dx"] = g["dx"].reshape(x.shape), m["dx"].reshape(x.shape)
    return {name: (g[name], m[name]) for name in g}


# ---------------------------------------------------------------------------
# RMS norms
# ---------------------------------------------------------------------------
def _rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def gated_norm(x, z, weight, eps=1e-6):
    """Returns (y, magnitude)."""
    x, z, w = f64(x), f64(z), f64(weight)
    y = x * _rms(x, eps) * w * z * sigmoid(z)
    return y, np.abs(y) * (1 + np.abs(z))


def gated_norm_bwd(x, z, weight, dy, eps=1e-6):
    """Returns {name: (gradient, magnitude)} for dx, dz, dweight."""
    x, z, w, dy = (f64(t) for t in (x, z, weight, dy))
    r, s = _rms(x, eps), sigmoid(z)
    n, silu, grow = x * r, z * s, 1 + np.abs(z)
    u = dy * w * silu
    c = (n * u).mean(-1, keepdims=True)
    mc = (np.abs(n * u) * grow).mean(-1, keepdims=True)
    rows = tuple(range(x.ndim - 1))
    return {"dx": (r * (u - n * c), r * (np.abs(u) * grow + np.abs(n) * mc)),
            "dz": (dy * n * w * s * (1 + z * (1 - s)), np.abs(dy * n * w) * s * (1 + np.abs(z) * (1 - s)) * grow),
            "dweight": ((dy * n * silu).sum(rows), (np.abs(dy * n * silu) * grow).sum(rows))}


def add_norm(x, residual, weight, eps=1e-6, residual_scale=1.0, weight_offset=0.0):
    """Returns (y, hidden)."""
    x, res, w = f64(x), f64(residual), f64(weight)
    h = residual_scale * x + (0 if res is None else res)
    return h * _rms(h, eps) * (w + weight_offset), h


def add_norm_bwd(dy, dhidden, hidden, weight, eps=1e-6, residual_scale=1.0, weight_offset=0.0):
    """Returns {name: (gradient, magnitude)} for dx, dresidual, dweight."""
    dy, dh, h, w = (f64(t) for t in (dy, dhidden, hidden, weight))
    w = w + weight_offset
    r = _rms(h, eps)
    n, u = h * r, dy * w
    c, mc = (n * u).mean(-1, keepdims=True), np.abs(n * u).mean(-1, keepdims=True)
    d = r * (u - n * c) + (0 if dh is None else dh)
    m = r * (np.abs(u) + np.abs(n) * mc) + (0 if dh is None else np.abs(dh))
    rows = tuple(range(h.ndim - 1))
    return {"dx": (residual_scale * d, abs(residual_scale) * m), "dresidual": (d, m),
            "dweight": ((dy * n).sum(rows), np.abs(dy * n).sum(rows))}
