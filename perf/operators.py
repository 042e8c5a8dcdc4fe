"""Timed cases of the operators around the chunked gated delta rule in a GDN layer.

A layer runs: residual add and RMS norm -> projections -> short causal
convolution of q, k, v -> the delta rule -> gated RMS norm -> output projection.
Beside the chunked pass the operators here are

  steps       the recurrent delta rule over a few tokens per sequence (a token and
              its drafts), states in a pool, the state after every token kept
  conv        the short causal convolution with SiLU over a (packed) batch
  conv_update the same for a few tokens per sequence, histories in a pool
  conv_bwd    its gradients
  gated_norm, gated_norm_bwd   RMS norm of the heads' outputs times SiLU(z)
  add_norm, add_norm_bwd       residual + scale * x, then RMS norm

``run`` makes the framework's calls where ``own`` is true and otherwise computes
the operators in plain torch, in 32 bits, rounded once at the end.  ``exact``
states the definitions again in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6          # of the RMS norms
L2_EPS = 1e-6       # of the L2 norm of q and k


def _device():
    return torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _steps(seqs, tokens, cols, ragged=False, H=16, HV=32, K=128, V=128, pool="fp32", gates=True, pad=0, dtype="bf16"):
    return {"op": "steps", "seqs": seqs, "tokens": tokens, "cols": cols, "ragged": ragged, "H": H, "HV": HV, "K": K,
            "V": V, "pool": pool, "gates": gates, "pad": pad, "dtype": dtype}


def _conv(op, seqs, tokens, q, v, ragged=False, width=4, bias=False, split=True, extra=0, cols=1, pad=0, dtype="bf16"):
    """q, v: the columns of q (and of k) and of v; extra: further columns of the projection that x is a slice of."""
    return {"op": op, "seqs": seqs, "tokens": tokens, "q": q, "v": v, "ragged": ragged, "width": width, "bias": bias,
            "split": split, "extra": extra, "cols": cols, "pad": pad, "dtype": dtype}


def _gated(op, tokens, heads, dim, extra=0, dtype="bf16"):
    return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "extra": extra, "dtype": dtype}


def _add(op, rows, dim, scale=1.0, offset=0.0, dtype="bf16"):
    return {"op": op, "rows": rows, "dim": dim, "scale": scale, "offset": offset, "dtype": dtype}


def listed():
    return [
        # one user, a token and three drafts to verify: latency
        {"name": "steps one user", **_steps(1, 4, 4)},
        # a batch of users with three drafts each, the state after every token kept, two padded rows
        {"name": "steps verify batch", **_steps(64, 4, 4, pad=2)},
        # 256 users, 0 to 8 tokens each (the remainders of prompts), one bf16 slot per user
        {"name": "steps ragged bf16 pool", **_steps(256, 8, 1, ragged=True, pool="bf16", gates=False, pad=8)},
        # the decode batch of 256 rows: one token each, its history in the pool
        {"name": "conv decode", **_conv("conv_update", 256, 1, 2048, 4096, pad=8)},
        # packed prompts of 1 to 2048 tokens; x is the q, k, v part of a projection that also holds z
        {"name": "conv packed prompts", **_conv("conv", 64, 2048, 2048, 4096, ragged=True, extra=4096)},
        # fp32, an odd length and width 3: the check mode on sizes without a vector's alignment
        {"name": "conv fp32 odd", **_conv("conv", 2, 1021, 0, 1001, width=3, bias=True, split=False, dtype="fp32")},
        # the training step of the grouped-value-head batch
        {"name": "conv backward", **_conv("conv_bwd", 4, 4096, 2048, 4096)},
        # a small decode batch: latency; z is a slice of the projection
        {"name": "gated norm decode", **_gated("gated_norm", 8, 32, 128, extra=8192)},
        # the training step of the grouped-value-head batch
        {"name": "gated norm backward", **_gated("gated_norm_bwd", 16384, 32, 128)},
        # the decode batch's hidden rows
        {"name": "add norm decode", **_add("add_norm", 256, 2048, offset=1.0)},
        # hidden rows of a prefill or training batch, with a residual scale
        {"name": "add norm rows", **_add("add_norm", 16384, 5120, scale=0.5)},
        # their gradients, at an odd number of rows
        {"name": "add norm backward", **_add("add_norm_bwd", 16383, 4096, scale=0.5, offset=1.0)},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["steps", "steps", "conv", "conv_update", "conv_bwd", "gated_norm", "gated_norm_bwd", "add_norm",
                     "add_norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "steps":
        H, G = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4])
        seqs, tokens = _log(rng, 1, 256), rng.randint(1, 8)
        c = _steps(seqs, tokens, rng.choice([1, tokens]), rng.random() < 0.5, H, H * G, rng.choice([64, 128]),
                   rng.choice([64, 128]), rng.choice(["fp32", "fp32", "bf16"]), rng.random() < 0.5,
                   rng.randint(0, seqs // 8), dtype)
        most, key = 7e8, "seqs"
    elif op.startswith("conv"):
        vec = 1 if rng.random() < 0.25 else 64
        q = vec * _log(rng, 1, 2048 // vec)
        v = vec * _log(rng, 1, 4096 // vec)
        if op == "conv_update":
            seqs, tokens = _log(rng, 1, 256), rng.randint(1, 8)
        else:
            seqs, tokens = _log(rng, 1, 64), _log(rng, 1, 8192)
        c = _conv(op, seqs, tokens, q, v, rng.random() < 0.5, rng.choice([2, 3, 4, 4, 4]), rng.random() < 0.5,
                  rng.random() < 0.7, rng.choice([0, v]), rng.choice([1, tokens]) if op == "conv_update" else 1,
                  rng.randint(0, seqs // 8) if op == "conv_update" else 0, dtype)
        most, key = 1.2e9, "tokens" if op != "conv_update" else "seqs"
    elif op.startswith("gated_norm"):
        c = _gated(op, _log(rng, 1, 32768), _log(rng, 1, 64), rng.choice([64, 128, 128, rng.randint(1, 256)]),
                   0, dtype)
        c["extra"] = rng.choice([0, c["heads"] * c["dim"]])
        most, key = 7e8, "tokens"
    else:
        c = _add(op, _log(rng, 1, 32768), rng.choice([256 * rng.randint(2, 32), _log(rng, 1, 8192)]),
                 rng.choice([1.0, round(rng.uniform(0.1, 2.0), 3)]), rng.choice([0.0, 1.0]), dtype)
        most, key = 7e8, "rows"
    while work(c)["bytes"] > most and c[key] > 1:
        c[key] = (c[key] + 1) // 2
        c["pad"] = min(c["pad"], c["seqs"] // 8) if "pad" in c else 0
        if "pad" in c and "seqs" not in c:
            del c["pad"]
    return c


def _lengths(c):
    """The sequences' lengths: the case's own, the same for every seed."""
    if not c["ragged"]:
        return [c["tokens"]] * c["seqs"]
    r = random.Random("%d sequences of up to %d tokens" % (c["seqs"], c["tokens"]))
    low = 0 if c["op"] in ("steps", "conv_update") else 1
    return [r.randint(low, c["tokens"]) for _ in range(c["seqs"] - 1)] + [c["tokens"]]


def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "steps":
        lens = _lengths(c)[c["pad"]:]                    # the first rows are padding: only their zeros are written
        T, Tall = sum(lens), sum(_lengths(c))
        se = 2 if c["pool"] == "bf16" else 4
        state = c["HV"] * c["K"] * c["V"]
        reads, writes = sum(n > 0 for n in lens), sum(min(n, c["cols"]) for n in lens)
        gate = 2 * c["HV"] * (e if c["gates"] else 4)
        return {"bytes": state * se * (reads + writes) + T * (2 * c["H"] * c["K"] * e + c["HV"] * c["V"] * e + gate)
                + Tall * c["HV"] * c["V"] * e + 4 * c["seqs"] * (c["cols"] + 1),
                "flops": T * state * 8}
    if c["op"].startswith("conv"):
        D, W, T = 2 * c["q"] + c["v"], c["width"], sum(_lengths(c))
        hist = D * (W - 1) * e
        n = c["seqs"]
        if c["op"] == "conv_bwd":
            return {"bytes": 3 * T * D * e + D * (W + 1) * (e + 4), "flops": T * D * (6 * W + 12)}
        live = [m for m in _lengths(c)[c["pad"]:] if m > 0]
        reads, writes = len(live), sum(min(m, c["cols"]) for m in live)
        return {"bytes": 2 * T * D * e + hist * (reads + writes) + D * (W + 1) * e + 4 * n, "flops": T * D * (2 * W + 5)}
    if c["op"].startswith("gated_norm"):
        n = c["tokens"] * c["heads"] * c["dim"]
        bwd = c["op"].endswith("bwd")
        return {"bytes": n * e * (5 if bwd else 3) + c["dim"] * (e + 4 * bwd), "flops": n * (24 if bwd else 10)}
    n = c["rows"] * c["dim"]
    bwd = c["op"].endswith("bwd")
    return {"bytes": n * e * (5 if bwd else 4) + c["dim"] * (e + 4 * bwd), "flops": n * (12 if bwd else 7)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    c, dev, dt = case, _device(), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dtype)

    def rand(*shape, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32) * hi

    s = {"case": dict(c)}
    if c["op"] == "steps" or c["op"].startswith("conv"):
        lens = _lengths(c)
        N, T = len(lens), sum(lens)
        s["longest"] = max(lens)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32).to(dev) if c["ragged"] else None
        B = 1 if c["ragged"] else N
        s["B"], s["T"], s["N"] = B, T // B, N
    if c["op"] in ("steps", "conv_update"):
        # slots in any order, the first `pad` rows padding; how many tokens of the step before were kept
        slots = N * c["cols"] + 3
        s["idx"] = torch.randperm(slots, generator=gen, device=dev)[:N * c["cols"]].to(torch.int32).view(N, c["cols"])
        s["idx"][:c["pad"]] = -1
        s["kept"] = torch.randint(1, c["cols"] + 1, (N,), generator=gen, device=dev, dtype=torch.int32)
    if c["op"] == "steps":
        H, HV, K, V = c["H"], c["HV"], c["K"], c["V"]
        s["q"], s["k"] = randn(B, s["T"], H, K), randn(B, s["T"], H, K)
        s["v"] = randn(B, s["T"], HV, V)
        s["A_log"], s["dt_bias"] = rand(HV, hi=math.log(16.0)), rand(HV)
        s["a"], s["b"] = randn(B, s["T"], HV), randn(B, s["T"], HV)
        if not c["gates"]:
            s["g"] = -s["A_log"].exp() * torch.nn.functional.softplus(s["a"].float() + s["dt_bias"])
            s["beta"] = s["b"].float().sigmoid()
        # one slot more than the pool has, where the plain form sends what is not kept
        s["store"] = randn(slots + 1, HV, K, V, std=0.05, dtype=DTYPES[c["pool"]])
        s["pool"] = s["store"][:slots]
    elif c["op"].startswith("conv"):
        D, W = 2 * c["q"] + c["v"], c["width"]
        wide = randn(B, s["T"], D + c["extra"])
        s["x"] = wide[..., :D]
        s["weight"], s["bias"] = randn(D, W, std=W ** -0.5), randn(D, std=0.2) if c["bias"] else None
        s["sizes"] = (c["q"], c["q"], c["v"]) if c["split"] and c["q"] else None
        if c["op"] == "conv_bwd":
            s["dy"] = [randn(B, s["T"], n) for n in s["sizes"] or (D,)]
        elif c["op"] == "conv_update":
            s["store"] = randn(slots + 1, D, W - 1)
            s["pool"] = s["store"][:slots]
        else:
            s["h0"] = randn(N, D, W - 1)
    elif c["op"].startswith("gated_norm"):
        t, h, d = c["tokens"], c["heads"], c["dim"]
        s["x"] = randn(t, h, d)
        s["z"] = randn(t, c["extra"] + h * d)[:, c["extra"]:].view(t, h, d)
        s["weight"] = randn(d, std=0.2) + 1
        if c["op"].endswith("bwd"):
            s["dy"] = randn(t, h, d)
    else:
        n, d = c["rows"], c["dim"]
        s["weight"] = randn(d, std=0.2) + (1 - c["offset"])
        s["h"] = randn(n, d, std=2.0)
        if c["op"].endswith("bwd"):
            s["dy"], s["dh"] = randn(n, d), randn(n, d)
        else:
            s["x"] = randn(n, d)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        return OWN[c["op"]](s, c)
    return PLAIN[c["op"]](s, c)


def own_steps(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    gates = {"A_log": s["A_log"], "dt_bias": s["dt_bias"], "a_raw": s["a"], "b_raw": s["b"]} if c["gates"] else {}
    out = gdn.fused_recurrent_gated_delta_rule_steps(
        s["q"], s["k"], s["v"], s.get("g"), s.get("beta"), s["pool"], s["idx"], cu_seqlens=s["cu"],
        num_accepted=s["kept"], use_qk_l2norm_in_kernel=True, **gates)
    return out, s["pool"]


def own_conv(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.causal_conv1d(s["x"], s["weight"], s["bias"], initial_state=s["h0"], cu_seqlens=s["cu"],
                             split_sizes=s["sizes"])


def own_conv_update(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.causal_conv1d_update(s["x"], s["weight"], s["pool"], s["idx"], s["bias"], cu_seqlens=s["cu"],
                                    num_accepted=s["kept"], split_sizes=s["sizes"]), s["pool"]


def own_conv_bwd(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    dx, dw, db, _ = gdn.causal_conv1d_bwd(s["x"], s["weight"], s["dy"] if s["sizes"] else s["dy"][0], s["bias"],
                                          cu_seqlens=s["cu"])
    return dx, dw, db


def own_gated_norm(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.fused_gated_rms_norm(s["x"], s["z"], s["weight"], eps=EPS)


def own_gated_norm_bwd(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.fused_gated_rms_norm_bwd(s["x"], s["z"], s["weight"], s["dy"], eps=EPS)


def own_add_norm(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.fused_add_rms_norm(s["x"], s["h"], s["weight"], eps=EPS, residual_scale=c["scale"],
                                  weight_offset=c["offset"])


def own_add_norm_bwd(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.fused_add_rms_norm_bwd(s["dy"], s["dh"], s["h"], s["weight"], eps=EPS, residual_scale=c["scale"],
                                      weight_offset=c["offset"])


OWN = {"steps": own_steps, "conv": own_conv, "conv_update": own_conv_update, "conv_bwd": own_conv_bwd,
       "gated_norm": own_gated_norm, "gated_norm_bwd": own_gated_norm_bwd, "add_norm": own_add_norm,
       "add_norm_bwd": own_add_norm_bwd}


def _starts(s):
    """First token and length of every sequence, on the device."""
    if s["cu"] is not None:
        cu = s["cu"].long()
        return cu[:-1], cu[1:] - cu[:-1]
    dev = s["x"].device if "x" in s else s["q"].device
    return torch.arange(s["N"], device=dev) * s["T"], torch.full((s["N"],), s["T"], device=dev)


def _places(s, start):
    """The sequence and the position in it of every token."""
    t = torch.arange(s["B"] * s["T"], device=start.device)
    ends = torch.cat([start[1:], start.new_full((1,), s["B"] * s["T"])])
    seq = (t[:, None] >= ends[None, :]).sum(1)
    return seq, t - start[seq]


def _first(s, c):
    """The slot that each row starts from, and whether it has one."""
    slot = s["idx"].long().gather(1, s["kept"].long()[:, None] - 1)[:, 0]
    return slot, (slot >= 0) & (slot < s["pool"].shape[0])


def plain_steps(s, c):
    H, HV, K, V = c["H"], c["HV"], c["K"], c["V"]
    start, length = _starts(s)
    seq, pos = _places(s, start)
    dt, total = s["q"].dtype, s["B"] * s["T"]
    q, k = (s[n].reshape(total, H, K).float() for n in "qk")
    q, k = (x * (x.square().sum(-1, keepdim=True) + L2_EPS).rsqrt() for x in (q, k))
    q, k = (x.repeat_interleave(HV // H, 1) for x in (q, k))
    v = s["v"].reshape(total, HV, V).float()
    if c["gates"]:
        x = s["a"].reshape(total, HV).float() + s["dt_bias"]
        g = -s["A_log"].exp() * (x.clamp(min=0) + (-x.abs()).exp().log1p())
        beta = 1 / (1 + (-s["b"].reshape(total, HV).float()).exp())
    else:
        g, beta = s["g"].reshape(total, HV), s["beta"].reshape(total, HV)
    slot, live = _first(s, c)
    S = s["pool"][slot.clamp(min=0)].float()
    spare, outs = s["pool"].shape[0], []
    for t in range(s["longest"]):       # the recurrence: a token's state needs the one before
        i = (start + t).clamp(max=max(total - 1, 0))
        S = S * g[i].exp()[..., None, None]
        u = beta[i][..., None] * (v[i] - (S * k[i][..., None]).sum(2))
        S = S + k[i][..., None] * u[:, :, None, :]
        outs.append((S * q[i][..., None]).sum(2) * K ** -0.5)
        # column t takes the state after token t + 1, the last column the one after the last token
        last = t + 1 == length
        keep = live & (t < length) & (last if t >= c["cols"] - 1 else torch.ones_like(last))
        to = s["idx"].long()[:, min(t, c["cols"] - 1)]
        to = torch.where(keep & (to >= 0), to, torch.full_like(to, spare))
        s["store"][to] = S.to(s["store"].dtype)
    o = torch.stack(outs)[pos, seq] * live[seq][:, None, None]
    return o.to(dt).view(s["v"].shape), s["pool"]


def _conv_rows(s, c, hist):
    """x with every sequence's history before it, as rows of one buffer; the row of a (sequence, position)."""
    W1, D = c["width"] - 1, s["x"].shape[-1]
    rows = torch.cat([hist.transpose(1, 2).reshape(s["N"] * W1, D), s["x"].reshape(-1, D)]).float()
    start, length = _starts(s)

    def row(seq, pos):
        return torch.where(pos < 0, seq * W1 + W1 + pos, s["N"] * W1 + start[seq] + pos)
    return rows, row, start, length


def _conv_pre(s, c, rows, row, seq, pos):
    w = s["weight"].float()
    pre = sum(rows[row(seq, pos - lag)] * w[:, c["width"] - 1 - lag] for lag in range(c["width"]))
    return pre if s["bias"] is None else pre + s["bias"].float()


def _conv_out(s, c, y):
    y = y.view(s["x"].shape)
    return [p.contiguous() for p in y.split(s["sizes"], -1)] if s["sizes"] else y


def plain_conv(s, c):
    rows, row, start, length = _conv_rows(s, c, s["h0"])
    seq, pos = _places(s, start)
    pre = _conv_pre(s, c, rows, row, seq, pos)
    y = (pre / (1 + (-pre).exp())).to(s["x"].dtype)
    back = torch.arange(c["width"] - 1, device=start.device) - (c["width"] - 1)
    every = torch.arange(s["N"], device=start.device)[:, None]
    final = rows[row(every, length[:, None] + back)].transpose(1, 2).to(s["x"].dtype).contiguous()
    return _conv_out(s, c, y), final


def plain_conv_update(s, c):
    slot, live = _first(s, c)
    rows, row, start, length = _conv_rows(s, c, s["pool"][slot.clamp(min=0)])
    seq, pos = _places(s, start)
    pre = _conv_pre(s, c, rows, row, seq, pos)
    y = (pre / (1 + (-pre).exp()) * live[seq][:, None]).to(s["x"].dtype)
    # the history after token n of a sequence, for each column
    col = torch.arange(c["cols"], device=start.device)
    n = torch.where(col == c["cols"] - 1, length[:, None], col + 1)
    back = torch.arange(c["width"] - 1, device=start.device) - (c["width"] - 1)
    every = torch.arange(s["N"], device=start.device)[:, None, None]
    keep = live[:, None] & (col < length[:, None]) & (s["idx"] >= 0)
    place = n.minimum(length[:, None])[..., None] + back
    hist = rows[row(every.expand_as(place), place)].transpose(2, 3).to(s["x"].dtype)
    to = torch.where(keep, s["idx"].long(), torch.full_like(s["idx"], s["pool"].shape[0]).long())
    s["store"][to.reshape(-1)] = hist.reshape(-1, *hist.shape[2:])
    return _conv_out(s, c, y), s["pool"]


def plain_conv_bwd(s, c):
    W, D = c["width"], s["x"].shape[-1]
    rows, row, start, length = _conv_rows(s, c, s["x"].new_zeros(s["N"], D, W - 1))
    seq, pos = _places(s, start)
    pre = _conv_pre(s, c, rows, row, seq, pos)
    sig = 1 / (1 + (-pre).exp())
    dpre = torch.cat(s["dy"], -1).reshape(-1, D).float() * sig * (1 + pre * (1 - sig))
    w, total = s["weight"].float(), s["B"] * s["T"]
    later = torch.arange(total, device=start.device)
    dx = sum(dpre[(later + lag).clamp(max=total - 1)] * (pos + lag < length[seq])[:, None] * w[:, W - 1 - lag]
             for lag in range(W))
    dw = torch.stack([(dpre * rows[row(seq, pos - lag)]).sum(0) for lag in reversed(range(W))], 1)
    return dx.to(s["x"].dtype).view(s["x"].shape), dw, dpre.sum(0) if c["bias"] else None


def plain_gated_norm(s, c):
    x, z, w = s["x"].float(), s["z"].float(), s["weight"].float()
    y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w * (z / (1 + (-z).exp()))
    return y.to(s["x"].dtype)


def plain_gated_norm_bwd(s, c):
    x, z, w, dy = s["x"].float(), s["z"].float(), s["weight"].float(), s["dy"].float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n, sig = x * r, 1 / (1 + (-z).exp())
    dn = dy * (z * sig)
    dz = dy * n * w * (sig * (1 + z * (1 - sig)))
    dw = (dn * n).sum((0, 1))
    dn = dn * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return dx.to(s["x"].dtype), dz.to(s["x"].dtype), dw


def plain_add_norm(s, c):
    h = s["h"].float() + s["x"].float() * c["scale"]
    y = h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * (s["weight"].float() + c["offset"])
    return y.to(s["x"].dtype), h.to(s["x"].dtype)


def plain_add_norm_bwd(s, c):
    h, w, dy = s["h"].float(), s["weight"].float() + c["offset"], s["dy"].float()
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = h * r
    dw = (dy * n).sum(0)
    dn = dy * w
    dh = s["dh"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return (dh * c["scale"]).to(s["h"].dtype), dh.to(s["h"].dtype), dw


PLAIN = {"steps": plain_steps, "conv": plain_conv, "conv_update": plain_conv_update, "conv_bwd": plain_conv_bwd,
         "gated_norm": plain_gated_norm, "gated_norm_bwd": plain_gated_norm_bwd, "add_norm": plain_add_norm,
         "add_norm_bwd": plain_add_norm_bwd}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, a sequence at a time; gradients by differentiating them
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    for name, t in s.items():
        if isinstance(t, torch.Tensor) and t.is_floating_point():
            s[name] = t.double()
    if "pool" in s:
        s["pool"] = s["pool"].clone()
    return EXACT[case["op"]](s, case)


def exact_steps(s, c):
    H, HV, K, V = c["H"], c["HV"], c["K"], c["V"]
    q, k = (torch.nn.functional.normalize(s[n].view(-1, H, K), dim=-1, eps=0) for n in "qk")
    # x / sqrt(|x|^2 + eps), from the unit vectors and the norms
    q, k = (u * (n2 / (n2 + L2_EPS)).sqrt() for u, n2 in
            ((q, s["q"].view(-1, H, K).pow(2).sum(-1, keepdim=True)), (k, s["k"].view(-1, H, K).pow(2).sum(-1, keepdim=True))))
    v = s["v"].view(-1, HV, V)
    if c["gates"]:
        decay = torch.exp(-torch.exp(s["A_log"]) * torch.nn.functional.softplus(s["a"].view(-1, HV) + s["dt_bias"]))
        beta = torch.sigmoid(s["b"].view(-1, HV))
    else:
        decay, beta = torch.exp(s["g"].view(-1, HV)), s["beta"].view(-1, HV)
    out, before, t0 = torch.zeros_like(v), s["pool"].clone(), 0
    idx, kept = s["idx"].tolist(), s["kept"].tolist()
    group = torch.arange(HV, device=v.device) // (HV // H)
    for n, length in enumerate(_lengths(c)):
        slots, t1 = idx[n], t0 + length
        if slots[kept[n] - 1] >= 0:
            S = before[slots[kept[n] - 1]]
            for j, t in enumerate(range(t0, t1)):
                kt, qt = k[t][group].unsqueeze(-1), q[t][group].unsqueeze(-2)
                old = decay[t].view(HV, 1, 1) * (kt.transpose(1, 2) @ S)
                S = decay[t].view(HV, 1, 1) * S + kt @ (beta[t].view(HV, 1, 1) * (v[t].unsqueeze(1) - old))
                out[t] = (qt @ S).squeeze(1) / math.sqrt(K)
                col = min(j, c["cols"] - 1)
                if slots[col] >= 0 and (col < c["cols"] - 1 or t == t1 - 1):
                    s["pool"][slots[col]] = S
        t0 = t1
    return out.view(s["v"].shape), s["pool"]


def _exact_conv(x, hist, weight, bias):
    """One sequence: x [T, D], hist [D, W-1] -> SiLU(conv) [T, D] and the row of inputs [D, W-1+T]."""
    line = torch.cat([hist, x.t()], 1)
    y = (line.unfold(1, weight.shape[1], 1) * weight[:, None, :]).sum(-1)
    return torch.nn.functional.silu(y if bias is None else y + bias[:, None]).t(), line


def _exact_split(s, y):
    y = y.view(s["x"].shape)
    return list(y.split(s["sizes"], -1)) if s["sizes"] else y


def exact_conv(s, c):
    x, at, ys, ends = s["x"].reshape(-1, s["x"].shape[-1]), 0, [], []
    for n, length in enumerate(_lengths(c)):
        y, line = _exact_conv(x[at:at + length], s["h0"][n], s["weight"], s["bias"])
        ys.append(y)
        ends.append(line[:, length:])
        at += length
    return _exact_split(s, torch.cat(ys)), torch.stack(ends)


def exact_conv_update(s, c):
    x, at, ys, before, W1 = s["x"].reshape(-1, s["x"].shape[-1]), 0, [], s["pool"].clone(), c["width"] - 1
    idx, kept = s["idx"].tolist(), s["kept"].tolist()
    for n, length in enumerate(_lengths(c)):
        if idx[n][kept[n] - 1] < 0:
            ys.append(torch.zeros_like(x[at:at + length]))
        else:
            if length:
                y, line = _exact_conv(x[at:at + length], before[idx[n][kept[n] - 1]], s["weight"], s["bias"])
                ys.append(y)
            for col in range(min(length, c["cols"])):
                n_in = length if col == c["cols"] - 1 else col + 1
                if idx[n][col] >= 0:
                    s["pool"][idx[n][col]] = line[:, n_in:n_in + W1]
        at += length
    return _exact_split(s, torch.cat(ys) if ys else x), s["pool"]


def exact_conv_bwd(s, c):
    D = s["x"].shape[-1]
    x, w = s["x"].reshape(-1, D).clone().requires_grad_(), s["weight"].clone().requires_grad_()
    b = s["bias"].clone().requires_grad_() if c["bias"] else None
    dy = torch.cat([d.double() for d in s["dy"]], -1).reshape(-1, D)
    at, none = 0, x.new_zeros(D, c["width"] - 1)
    for length in _lengths(c):
        _exact_conv(x[at:at + length], none, w, b)[0].backward(dy[at:at + length])
        at += length
    return x.grad.view(s["x"].shape), w.grad, b.grad if c["bias"] else None


def _exact_gated(x, z, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w * torch.nn.functional.silu(z)


def exact_gated_norm(s, c):
    return _exact_gated(s["x"], s["z"], s["weight"])


def exact_gated_norm_bwd(s, c):
    x, z, w = (s[n].clone().requires_grad_() for n in ("x", "z", "weight"))
    _exact_gated(x, z, w).backward(s["dy"])
    return x.grad, z.grad, w.grad


def exact_add_norm(s, c):
    h = s["h"] + c["scale"] * s["x"]
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * (s["weight"] + c["offset"]), h


def exact_add_norm_bwd(s, c):
    h, w = s["h"].clone().requires_grad_(), s["weight"].clone().requires_grad_()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * (w + c["offset"])
    torch.autograd.backward([y, h], [s["dy"], s["dh"]])
    return c["scale"] * h.grad, h.grad, w.grad


EXACT = {"steps": exact_steps, "conv": exact_conv, "conv_update": exact_conv_update, "conv_bwd": exact_conv_bwd,
         "gated_norm": exact_gated_norm, "gated_norm_bwd": exact_gated_norm_bwd, "add_norm": exact_add_norm,
         "add_norm_bwd": exact_add_norm_bwd}
