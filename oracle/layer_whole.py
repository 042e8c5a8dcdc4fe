"""The float64 definitions of oracle/layer.py over whole torch tensors, on the
device the inputs are on: for sizes where loops over tokens take minutes.  The
magnitudes are those of oracle/layer.py.  Sequences are given as a list of lengths.
"""
from __future__ import annotations

import torch


def _taps(x, hist, lens, W):
    """x [T, D], hist [N, D, W-1]: the W rows that each token's output reads, oldest first, and each token's
    sequence, position and its sequence's length."""
    n = torch.tensor(lens, device=x.device)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=x.device), n)
    start = n.cumsum(0) - n
    pos = torch.arange(x.shape[0], device=x.device) - start[seq]
    rows = []
    for j in range(W):
        lag = W - 1 - j
        r = torch.roll(x, lag, 0)
        early = (pos < lag).nonzero()[:, 0]
        r[early] = hist[seq[early], :, j + pos[early]]    # row pos + j of the history with the sequence behind it
        rows.append(r)
    return rows, seq, pos, n[seq]


def _pre(rows, w, b):
    pre, size = torch.zeros_like(rows[0]), torch.zeros_like(rows[0])
    for j, r in enumerate(rows):
        pre += r * w[:, j]
        size += r.abs() * w[:, j].abs()
    return (pre, size) if b is None else (pre + b, size + b.abs())


def _inputs(x, weight, bias, initial, lens):
    x, w = x.reshape(-1, x.shape[-1]).double(), weight.double()
    D, W = w.shape
    hist = x.new_zeros(len(lens), D, W - 1) if initial is None else initial.double()
    return x, w, None if bias is None else bias.double(), hist, D, W


def conv(x, weight, bias, initial, lens, silu=True):
    """Returns (y [T, D], final_state, magnitude of y)."""
    x, w, b, hist, D, W = _inputs(x, weight, bias, initial, lens)
    rows, seq, pos, n = _taps(x, hist, lens, W)
    pre, size = _pre(rows, w, b)
    y = pre * torch.sigmoid(pre) if silu else pre
    final = hist.clone()
    last = (pos == n - 1).nonzero()[:, 0]
    for j in range(1, W):
        final[seq[last], :, j - 1] = rows[j][last]
    return y, final, 1.1 * size + y.abs() * (1 + pre.abs())


def conv_bwd(x, weight, dy, bias, initial, lens, silu=True):
    """Returns {name: (gradient, magnitude)} for dx, dweight, dbias, dinitial."""
    x, w, b, hist, D, W = _inputs(x, weight, bias, initial, lens)
    dy = dy.reshape(-1, D).double()
    rows, seq, pos, n = _taps(x, hist, lens, W)
    pre, size = _pre(rows, w, b)
    s = torch.sigmoid(pre)
    d = {0: dy * (s * (1 + pre * (1 - s)) if silu else 1.0),                          # the gradient of pre,
         1: 1.2 * dy.abs() * (1 + size + pre.abs()) * (1 + pre.abs())}                # and its magnitude
    out = {}
    for i, weights in ((0, w), (1, w.abs())):
        dx, dini = torch.zeros_like(x), torch.zeros_like(hist)
        for j in range(W):
            lag = W - 1 - j
            dx += torch.roll(d[i], -lag, 0) * (pos + lag < n)[:, None] * weights[:, j]
            # the token at position p reads row p + j of the history with its sequence behind it
            for p in range(W - 1 - j):
                at = (pos == p).nonzero()[:, 0]
                dini[seq[at], :, p + j] += d[i][at] * weights[:, j]
        out[i] = {"dx": dx, "dweight": torch.stack([(d[i] * (r.abs() if i else r)).sum(0) for r in rows], 1),
                  "dbias": d[i].sum(0), "dinitial": dini}
    return {name: (out[0][name], out[1][name]) for name in out[0]}


def _rms(x, eps):
    return (x.square().mean(-1, keepdim=True) + eps).rsqrt()


def gated_norm(x, z, weight, eps=1e-6):
    """Returns (y, magnitude)."""
    x, z, w = x.double(), z.double(), weight.double()
    y = x * _rms(x, eps) * w * z * torch.sigmoid(z)
    return y, y.abs() * (1 + z.abs())


def gated_norm_bwd(x, z, weight, dy, eps=1e-6):
    """Returns {name: (gradient, magnitude)} for dx, dz, dweight."""
    x, z, w, dy = x.double(), z.double(), weight.double(), dy.double()
    r, s = _rms(x, eps), torch.sigmoid(z)
    n, silu, grow = x * r, z * s, 1 + z.abs()
    u = dy * w * silu
    c, mc = (n * u).mean(-1, keepdim=True), ((n * u).abs() * grow).mean(-1, keepdim=True)
    rows = tuple(range(x.dim() - 1))
    return {"dx": (r * (u - n * c), r * (u.abs() * grow + n.abs() * mc)),
            "dz": (dy * n * w * s * (1 + z * (1 - s)), (dy * n * w).abs() * s * (1 + z.abs() * (1 - s)) * grow),
            "dweight": ((dy * n * silu).sum(rows), ((dy * n * silu).abs() * grow).sum(rows))}


def add_norm(x, residual, weight, eps=1e-6, residual_scale=1.0, weight_offset=0.0):
    """Returns (y, hidden, magnitude of y, magnitude of hidden): hidden may cancel, so its error is a share of its
    terms' size and y has that times r |weight + offset|."""
    x, w = x.double(), weight.double() + weight_offset
    res = torch.zeros_like(x) if residual is None else residual.double()
    h = res + residual_scale * x
    size = res.abs() + abs(residual_scale) * x.abs()
    r = _rms(h, eps)
    y = h * r * w
    return y, h, y.abs() + size * w.abs() * r, size


def add_norm_bwd(dy, dhidden, hidden, weight, eps=1e-6, residual_scale=1.0, weight_offset=0.0):
    """Returns {name: (gradient, magnitude)} for dx, dresidual, dweight."""
    dy, h, w = dy.double(), hidden.double(), weight.double() + weight_offset
    dh = torch.zeros_like(h) if dhidden is None else dhidden.double()
    r = _rms(h, eps)
    n, u = h * r, dy * w
    c, mc = (n * u).mean(-1, keepdim=True), (n * u).abs().mean(-1, keepdim=True)
    d = r * (u - n * c) + dh
    m = r * (u.abs() + n.abs() * mc) + dh.abs()
    rows = tuple(range(h.dim() - 1))
    return {"dx": (residual_scale * d, abs(residual_scale) * m), "dresidual": (d, m),
            "dweight": ((dy * n).sum(rows), (dy * n).abs().sum(rows))}
