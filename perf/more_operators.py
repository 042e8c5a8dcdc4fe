"""Timed cases of the gated linear recurrence and of the 8 and 4 bit memories of recurrent layers.

  rec, rec_bwd   h_t = e^(g_t) h_(t-1) + beta_t x_t per channel over a (packed) batch, and its gradients
  rec_steps      the same over a few tokens per sequence (a token and its drafts), states in a pool
  cache          states written into a cache of 8 or 4 bits and read back into a pool
  norm_step      the gated RMS norm that keeps its inputs in 8 bits, and its gradients from them
  norm_bwd       those gradients alone

What is held in 8 or 4 bits: groups of 32 along the last axis (of the whole slot in a
cache).  With top = 127 or 7, a group's scale s is the smallest bfloat16 that has
top * s >= the group's largest magnitude, and 0 where that is below 2^-100; a value's
code is the integer nearest to value / s, ties to even; it stands for code * s.

``run`` makes the framework's calls where ``own`` is true and otherwise computes the
operators in plain torch, in 32 bits, rounded once at the end.  ``exact`` states the
definitions again in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6          # of the RMS norm
GROUP = 32          # elements of one scale
TINY = 2.0 ** -100


def _device():
    return torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _rec(op, seqs, tokens, D, ragged=False, gate="fp32", beta=True, dtype="bf16", bits8=False, extra=0):
    """extra: further columns of the projection that x is a slice of; bits8: x and y are kept in 8 bits."""
    return {"op": op, "seqs": seqs, "tokens": tokens, "D": D, "ragged": ragged, "gate": gate, "beta": beta,
            "dtype": dtype, "bits8": bits8, "extra": extra}


def _steps(seqs, tokens, cols, D, ragged=False, gate="fp32", beta=True, pool="fp32", pad=0, dtype="bf16"):
    return {"op": "rec_steps", "seqs": seqs, "tokens": tokens, "cols": cols, "D": D, "ragged": ragged, "gate": gate,
            "beta": beta, "pool": pool, "pad": pad, "dtype": dtype}


def _cache(slots, heads, rows, cols, bits, pool="fp32"):
    return {"op": "cache", "slots": slots, "heads": heads, "rows": rows, "cols": cols, "bits": bits, "pool": pool}


def _norm(op, tokens, heads, dim, extra=0, dtype="bf16"):
    return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "extra": extra, "dtype": dtype}


def listed():
    return [
        # one user, a token and three drafts to verify: latency
        {"name": "recurrence one user", **_steps(1, 4, 4, 4096)},
        # a batch of users with three drafts each, the state after every token kept, two padded rows
        {"name": "recurrence verify batch", **_steps(64, 4, 4, 4096, pad=2)},
        # packed prompts of 1 to 2048 tokens, gates as the gating operator writes them
        {"name": "recurrence packed prompts", **_rec("rec", 64, 2048, 4096, ragged=True, extra=4096)},
        # one long prompt, bf16 gates, inputs scaled by the caller
        {"name": "recurrence long", **_rec("rec", 1, 131072, 4096, gate="bf16", beta=False)},
        # fp32, an odd length and an odd number of channels
        {"name": "recurrence fp32 odd", **_rec("rec", 2, 1021, 1001, dtype="fp32")},
        # a training step's batch
        {"name": "recurrence backward", **_rec("rec_bwd", 4, 4096, 4096)},
        # packed training sequences, x and y kept in 8 bits
        {"name": "recurrence backward 8 bit", **_rec("rec_bwd", 64, 2048, 4096, ragged=True, gate="bf16", bits8=True)},
        # one request's delta-rule state, swapped out and in
        {"name": "cache one state", **_cache(1, 32, 128, 128, 8)},
        # a batch of delta-rule states in a prefix cache
        {"name": "cache states 4 bit", **_cache(256, 32, 128, 128, 4, pool="bf16")},
        # the convolution histories beside them
        {"name": "cache histories", **_cache(64, 1, 8192, 3, 8, pool="bf16")},
        # the training step of the grouped-value-head batch: forward, then the gradients
        {"name": "norm step", **_norm("norm_step", 16384, 32, 128)},
        # the gradients alone, rows without a whole number of groups, z a slice of the projection
        {"name": "norm backward odd", **_norm("norm_bwd", 2047, 16, 100, extra=1600)},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rec", "rec", "rec_bwd", "rec_bwd", "rec_steps", "cache", "cache", "norm_step", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    gate = rng.choice(["fp32", dtype])
    D = _log(rng, 1, 8192) if rng.random() < 0.3 else 64 * _log(rng, 1, 128)
    if op == "rec_steps":
        seqs, tokens = _log(rng, 1, 256), rng.randint(1, 8)
        c = _steps(seqs, tokens, rng.choice([1, tokens]), D, rng.random() < 0.5, gate, rng.random() < 0.5,
                   rng.choice(["fp32", "fp32", "bf16"]), rng.randint(0, seqs // 8), dtype)
        most, key = 7e8, "seqs"
    elif op.startswith("rec"):
        bits8 = op == "rec_bwd" and rng.random() < 0.4
        c = _rec(op, _log(rng, 1, 64), _log(rng, 1, 131072), D, rng.random() < 0.5, gate, rng.random() < 0.6, dtype,
                 bits8, 0 if bits8 else rng.choice([0, D]))
        most, key = 2e9, "tokens"
    elif op == "cache":
        if rng.random() < 0.5:
            shape = (2 ** rng.randint(0, 5), rng.choice([64, 128]), rng.choice([64, 128]))
        else:
            shape = (1, _log(rng, 1, 16384), rng.choice([1, 3]))
        c = _cache(_log(rng, 1, 512), *shape, rng.choice([8, 4]), rng.choice(["fp32", "bf16"]))
        most, key = 5e8, "slots"
    else:
        c = _norm(op, _log(rng, 1, 32768), _log(rng, 1, 64), rng.choice([64, 128, 128, rng.randint(1, 256)]), 0, dtype)
        c["extra"] = rng.choice([0, c["heads"] * c["dim"]])
        most, key = 9e8, "tokens"
    while work(c)["bytes"] > most and c[key] > 1:
        c[key] = (c[key] + 1) // 2
        if "pad" in c:
            c["pad"] = min(c["pad"], c["seqs"] // 8)
    return c


def _lengths(c):
    """The sequences' lengths: the case's own, the same for every seed."""
    if not c["ragged"]:
        return [c["tokens"]] * c["seqs"]
    r = random.Random("%d sequences of up to %d tokens" % (c["seqs"], c["tokens"]))
    low = 0 if c["op"] == "rec_steps" else 1
    return [r.randint(low, c["tokens"]) for _ in range(c["seqs"] - 1)] + [c["tokens"]]


def _held(n, bits):
    return n * (bits / 8 + 2 / GROUP)


def work(case):
    c = case
    size = {"bf16": 2, "fp32": 4}
    if c["op"] == "rec_steps":
        e, ge, D = size[c["dtype"]], size[c["gate"]], c["D"]
        lens = _lengths(c)[c["pad"]:]            # the first rows are padding: only their zeros are written
        T, Tall = sum(lens), sum(_lengths(c))
        reads, writes = sum(n > 0 for n in lens), sum(min(n, c["cols"]) for n in lens)
        return {"bytes": D * (size[c["pool"]] * (reads + writes) + T * (e + ge * (1 + c["beta"])) + Tall * e)
                + 4 * c["seqs"] * (c["cols"] + 1), "flops": 4 * T * D}
    if c["op"].startswith("rec"):
        e, ge, D, T = size[c["dtype"]], size[c["gate"]], c["D"], sum(_lengths(c))
        kept = _held(1, 8) if c["bits8"] else e
        gates = ge * (1 + c["beta"])
        if c["op"] == "rec":                     # x, gates, y; the states
            return {"bytes": T * D * (2 * e + gates) + 8 * c["seqs"] * D, "flops": 4 * T * D}
        each = 2 * gates + 2 * e + kept * (1 + c["beta"])   # gates and their gradients, dy, dx, y (and x)
        return {"bytes": T * D * each + 12 * c["seqs"] * D, "flops": 9 * T * D}
    if c["op"] == "cache":
        n = c["slots"] * c["heads"] * c["rows"] * c["cols"]
        return {"bytes": 2 * n * size[c["pool"]] + 2 * _held(n, c["bits"]), "flops": 5 * n}
    n, e = c["tokens"] * c["heads"] * c["dim"], size[c["dtype"]]
    if c["op"] == "norm_step":
        return {"bytes": 6 * n * e + 4 * _held(n, 8) + c["dim"] * (2 * e + 4), "flops": 42 * n}
    return {"bytes": 3 * n * e + 2 * _held(n, 8) + c["dim"] * (e + 4), "flops": 26 * n}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    c, dev = case, _device()
    dt = DTYPES[c.get("dtype", "bf16")]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32)

    s = {"case": dict(c)}
    if c["op"].startswith("rec"):
        lens = _lengths(c)
        N, total, D, gt = len(lens), sum(lens), c["D"], DTYPES[c["gate"]]
        s["N"], s["total"], s["longest"] = N, total, max(lens)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32).to(dev) if c["ragged"] else None
        B = 1 if c["ragged"] else N
        shape = (B, total // B, D)
        # channels that forget within a few tokens and channels that keep hundreds
        rate = torch.exp(rand(D) * math.log(400.0)) * 0.005
        s["g"] = (-rate * torch.nn.functional.softplus(randn(*shape, dtype=torch.float32))).to(gt)
        s["beta"] = rand(*shape).to(gt) if c["beta"] else None
        s["x"] = randn(*shape[:2], D + c.get("extra", 0))[..., :D]
    if c["op"] == "rec_steps":
        # slots in any order, the first `pad` rows padding; how many tokens of the step before were kept
        slots = N * c["cols"] + 3
        s["idx"] = torch.randperm(slots, generator=gen, device=dev)[:N * c["cols"]].to(torch.int32).view(N, c["cols"])
        s["idx"][:c["pad"]] = -1
        s["kept"] = torch.randint(1, c["cols"] + 1, (N,), generator=gen, device=dev, dtype=torch.int32)
        # one slot more than the pool has, where the plain form sends what is not kept
        s["store"] = randn(slots + 1, D, dtype=DTYPES[c["pool"]])
        s["pool"] = s["store"][:slots]
    elif c["op"] == "rec":
        s["h0"] = randn(N, D, dtype=torch.float32)
    elif c["op"] == "rec_bwd":
        s["h0"], s["dht"] = randn(N, D, dtype=torch.float32), randn(N, D, dtype=torch.float32)
        s["dy"] = randn(*shape)
        s["y"] = plain_rec(s, c)[0]
        if c["bits8"]:
            s["y8"] = _quantise(s["y"].float(), 127)
            s["x8"] = _quantise(s["x"].float(), 127)
            s["x"] = s["y"] = None
    elif c["op"] == "cache":
        n, shape = c["slots"], (c["heads"], c["rows"], c["cols"])
        size, dt = math.prod(shape), DTYPES[c["pool"]]
        s["pool"] = randn(n + 3, *shape, dtype=dt)
        s["pool"] *= rand(n + 3, c["heads"], 1, 1) + 0.1
        s["back"] = torch.zeros_like(s["pool"])
        order = lambda m: torch.randperm(m, generator=gen, device=dev)[:n].to(torch.int32)  # noqa: E731
        s["from"], s["to"], s["at"] = order(n + 3), order(n + 3), order(n + 1)
        if c["bits"] == 8:
            s["codes"] = torch.zeros(n + 1, size, dtype=torch.int8, device=dev)
        else:
            s["codes"] = torch.zeros(n + 1, (size + 1) // 2, dtype=torch.uint8, device=dev)
        s["scales"] = torch.zeros(n + 1, -(-size // GROUP), dtype=torch.bfloat16, device=dev)
    elif c["op"].startswith("norm"):
        t, h, d = c["tokens"], c["heads"], c["dim"]
        s["x"] = randn(t, h, d)
        s["z"] = randn(t, c["extra"] + h * d)[:, c["extra"]:].view(t, h, d)
        s["weight"] = randn(d, std=0.2) + 1
        s["dy"] = randn(t, h, d)
        if c["op"] == "norm_bwd":
            s["x8"], s["z8"] = _quantise(s["x"].float(), 127), _quantise(s["z"].float(), 127)
            s["x"] = s["z"] = None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        return OWN[c["op"]](s, c)
    return PLAIN[c["op"]](s, c)


def own_rec(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.gated_linear_recurrence(s["x"], s["g"], s["beta"], initial_state=s["h0"], cu_seqlens=s["cu"])


def own_rec_steps(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.gated_linear_recurrence_steps(s["x"], s["g"], s["pool"], s["idx"], beta=s["beta"], cu_seqlens=s["cu"],
                                             num_accepted=s["kept"]), s["pool"]


def own_rec_bwd(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    x, y = (gdn.Checkpoint(*s["x8"]), gdn.Checkpoint(*s["y8"])) if c["bits8"] else (s["x"], s["y"])
    return gdn.gated_linear_recurrence_bwd(x, s["g"], y, s["dy"], s["beta"], dht=s["dht"], initial_state=s["h0"],
                                           cu_seqlens=s["cu"], output_dinitial=True)


def own_cache(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.state_cache_write(s["pool"], s["from"], s["codes"], s["scales"], s["at"])
    gdn.state_cache_read(s["codes"], s["scales"], s["at"], s["back"], s["to"])
    return s["back"]


def own_norm_step(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    y, x8, z8 = gdn.fused_gated_rms_norm_checkpoint(s["x"], s["z"], s["weight"], eps=EPS)
    return y, *gdn.fused_gated_rms_norm_checkpoint_bwd(x8, z8, s["weight"], s["dy"], eps=EPS)


def own_norm_bwd(s, c):
    import gated_deltanet_chunked_delta_amd as gdn
    return gdn.fused_gated_rms_norm_checkpoint_bwd(gdn.Checkpoint(*s["x8"]), gdn.Checkpoint(*s["z8"]), s["weight"],
                                                   s["dy"], eps=EPS)


OWN = {"rec": own_rec, "rec_steps": own_rec_steps, "rec_bwd": own_rec_bwd, "cache": own_cache,
       "norm_step": own_norm_step, "norm_bwd": own_norm_bwd}


def _grouped(v):
    """v [..., D] as [..., groups, 32], zeros behind a row's end."""
    short = -v.shape[-1] % GROUP
    return torch.nn.functional.pad(v, (0, short)).unflatten(-1, (-1, GROUP))


def _quantise(v, top):
    """v [..., D] fp32 -> codes int8 [..., D] and scales bf16 [..., groups]."""
    rows = _grouped(v)
    high = rows.abs().amax(-1)
    bits = (high / top).to(torch.bfloat16).view(torch.int16)
    # the neighbour below, the rounded one, or the one above: the smallest that reaches
    below = (bits - 1).clamp(min=0).view(torch.bfloat16)
    scale = torch.where(below.float() * top >= high, below, bits.view(torch.bfloat16))
    scale = torch.where(scale.float() * top < high, (bits + 1).view(torch.bfloat16), scale)
    scale = torch.where(high < TINY, torch.zeros_like(scale), scale)
    # in 64 bits: the quotients next to a border
    codes = (rows.double() / scale.double().masked_fill(scale == 0, math.inf)[..., None]).round().to(torch.int8)
    return codes.flatten(-2)[..., :v.shape[-1]].contiguous(), scale


def _values(codes, scales):
    rows = _grouped(codes).float() * scales.float()[..., None]
    return rows.flatten(-2)[..., :codes.shape[-1]]


def _starts(s):
    """First token and length of every sequence, on the device."""
    if s["cu"] is not None:
        cu = s["cu"].long()
        return cu[:-1], cu[1:] - cu[:-1]
    dev, T = s["g"].device, s["total"] // s["N"]
    return torch.arange(s["N"], device=dev) * T, torch.full((s["N"],), T, device=dev)


def _scan(a, u, longest):
    """h_t = a_t h_(t-1) + u_t along the first axis; a is 0 where a sequence begins, none is longer than `longest`."""
    step = 1
    while step < longest:       # each round doubles the tokens that a sum spans
        u = torch.cat([u[:step], u[step:] + a[step:] * u[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return u


def _rec_states(s, h0):
    """The recurrence's states, flat, from each sequence's h0; the sequences' starts and lengths."""
    D = s["g"].shape[-1]
    start, length = _starts(s)
    some = length > 0
    a, u = s["g"].float().exp().reshape(-1, D), s["x"].float()
    u = (u if s["beta"] is None else u * s["beta"].float()).reshape(-1, D)
    first = start[some]
    u = u.index_put((first,), u[first] + a[first] * h0[some])
    return _scan(a.index_fill(0, first, 0.0), u, s["longest"]), start, length


def plain_rec(s, c):
    h, start, length = _rec_states(s, s["h0"])
    return h.to(s["x"].dtype).view(s["g"].shape), h[start + length - 1]


def plain_rec_steps(s, c):
    slot = s["idx"].long().gather(1, s["kept"].long()[:, None] - 1)[:, 0]
    live = (slot >= 0) & (slot < s["pool"].shape[0])
    h, start, length = _rec_states(s, s["pool"][slot.clamp(min=0)].float())
    seq = torch.repeat_interleave(torch.arange(s["N"], device=h.device), length, output_size=s["total"])
    y = (h * live[seq][:, None]).to(s["x"].dtype).view(s["g"].shape)
    # column j takes the state after token j + 1, the last column the one after the last token
    col = torch.arange(c["cols"], device=h.device)
    n = torch.where(col == c["cols"] - 1, length[:, None], col + 1)
    keep = live[:, None] & (col < length[:, None]) & (s["idx"] >= 0)
    at = (start[:, None] + n - 1).clamp(0, max(s["total"] - 1, 0))
    to = torch.where(keep, s["idx"].long(), torch.full_like(s["idx"], s["pool"].shape[0]).long())
    s["store"][to.reshape(-1)] = h[at.reshape(-1)].to(s["store"].dtype)
    return y, s["pool"]


def plain_rec_bwd(s, c):
    shape, D = s["g"].shape, s["g"].shape[-1]
    y = (_values(*s["y8"]) if c["bits8"] else s["y"].float()).reshape(-1, D)
    start, length = _starts(s)
    last = start + length - 1
    a = s["g"].float().exp().reshape(-1, D)
    u = s["dy"].float().reshape(-1, D)
    u = u.index_put((last,), u[last] + s["dht"])
    later = torch.cat([a[1:], a[:1]]).index_fill(0, last, 0.0)
    dh = _scan(later.flip(0), u.flip(0), s["longest"]).flip(0)
    before = torch.cat([y[:1], y[:-1]]).index_put((start,), s["h0"])
    dg = a * before * dh
    dx, dbeta = dh, None
    if c["beta"]:
        x = (_values(*s["x8"]) if c["bits8"] else s["x"].float()).reshape(-1, D)
        dx, dbeta = s["beta"].float().reshape(-1, D) * dh, (x * dh).to(s["beta"].dtype).view(shape)
    return dx.to(s["dy"].dtype).view(shape), dg.to(s["g"].dtype).view(shape), dbeta, a[start] * dh[start]


def plain_cache(s, c):
    n, size, at = c["slots"], s["pool"][0].numel(), s["at"].long()
    codes, scales = _quantise(s["pool"][s["from"].long()].view(n, size).float(), 127 if c["bits"] == 8 else 7)
    if c["bits"] == 4:
        two = torch.nn.functional.pad(codes, (0, size % 2)).view(n, -1, 2) & 15
        codes = (two[..., 0] | two[..., 1] << 4).view(torch.uint8)
    s["codes"][at], s["scales"][at] = codes, scales
    codes = s["codes"][at]
    if c["bits"] == 4:
        two = torch.stack([codes & 15, codes >> 4], -1).to(torch.int8)
        codes = (two - (two > 7) * 16).view(n, -1)[:, :size]
    s["back"][s["to"].long()] = _values(codes, s["scales"][at]).to(s["back"].dtype).view(n, *s["back"].shape[1:])
    return s["back"]


def _norm_grads(x, z, w, dy):
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n, sig = x * r, 1 / (1 + (-z).exp())
    dn = dy * (z * sig)
    dz = dy * n * w * (sig * (1 + z * (1 - sig)))
    dw = (dn * n).sum((0, 1))
    dn = dn * w
    return r * (dn - n * (dn * n).mean(-1, keepdim=True)), dz, dw


def plain_norm_step(s, c):
    x, z, w = s["x"].float(), s["z"].float(), s["weight"].float()
    y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w * (z / (1 + (-z).exp()))
    dx, dz, dw = _norm_grads(_values(*_quantise(x, 127)), _values(*_quantise(z, 127)), w, s["dy"].float())
    return y.to(s["x"].dtype), dx.to(s["x"].dtype), dz.to(s["x"].dtype), dw


def plain_norm_bwd(s, c):
    dx, dz, dw = _norm_grads(_values(*s["x8"]), _values(*s["z8"]), s["weight"].float(), s["dy"].float())
    return dx.to(s["dy"].dtype), dz.to(s["dy"].dtype), dw


PLAIN = {"rec": plain_rec, "rec_steps": plain_rec_steps, "rec_bwd": plain_rec_bwd, "cache": plain_cache,
         "norm_step": plain_norm_step, "norm_bwd": plain_norm_bwd}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, a sequence at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rec", "rec_bwd") and sum(_lengths(case)) > 300000:
        return None     # one token after the other: more than 20 seconds
    return EXACT[case["op"]](s, case)


def _exact_round(v, top):
    """The values that v stands for after being held with magnitudes up to top."""
    v = v.double()
    out = torch.zeros_like(v)
    D = v.shape[-1]
    whole = D // GROUP * GROUP
    for part, to in ((v[..., :whole].unflatten(-1, (whole // GROUP, GROUP)), out[..., :whole]),
                     (v[..., None, whole:], out[..., whole:])):
        if part.numel() == 0:
            continue
        high = part.abs().max(-1, keepdim=True).values
        m, e = torch.frexp(high / torch.full_like(high, top))   # 8 significant bits, upwards
        s = torch.ceil(m * 256) * ((e.long() - 8 + 1023) << 52).view(torch.float64)
        q = part / torch.where(high < TINY, torch.inf, s)
        near = torch.floor(q + 0.5)
        near = torch.where((near - q == 0.5) & (near % 2 != 0), near - 1, near)
        to.copy_((near * torch.where(high < TINY, 0.0, s)).reshape(to.shape))
    return out


def _exact_held(pair):
    codes, scales = pair
    of = torch.arange(codes.shape[-1], device=codes.device) // GROUP
    return codes.double() * scales.double()[..., of]


def exact_rec(s, c):
    D = c["D"]
    a = torch.exp(s["g"].double()).reshape(-1, D)
    y = s["x"].double() if s["beta"] is None else s["x"].double() * s["beta"].double()
    y, at, ends = y.reshape(-1, D).contiguous(), 0, []
    for n, length in enumerate(_lengths(c)):
        h = s["h0"][n].double()
        for t in range(at, at + length):
            h = torch.addcmul(y[t], a[t], h, out=y[t])
        ends.append(h.clone())
        at += length
    return y.view(s["g"].shape), torch.stack(ends)


def exact_rec_steps(s, c):
    D = c["D"]
    a, x = torch.exp(s["g"].double()).reshape(-1, D), s["x"].double().reshape(-1, D)
    if s["beta"] is not None:
        x = x * s["beta"].double().reshape(-1, D)
    y, before, pool, at = torch.zeros_like(x), s["pool"].double(), s["pool"].double(), 0
    idx, kept = s["idx"].tolist(), s["kept"].tolist()
    for n, length in enumerate(_lengths(c)):
        if idx[n][kept[n] - 1] >= 0:
            h = before[idx[n][kept[n] - 1]]
            for j in range(length):
                h = a[at + j] * h + x[at + j]
                y[at + j] = h
                col = min(j, c["cols"] - 1)
                if idx[n][col] >= 0 and (col < c["cols"] - 1 or j == length - 1):
                    pool[idx[n][col]] = h
        at += length
    return y.view(s["g"].shape), pool


def exact_rec_bwd(s, c):
    shape, D = s["g"].shape, c["D"]
    a, dh = torch.exp(s["g"].double()).reshape(-1, D), s["dy"].double().reshape(-1, D).clone()
    y = (_exact_held(s["y8"]) if c["bits8"] else s["y"].double()).reshape(-1, D)
    dg, dh0, at = torch.empty_like(a), [], 0
    for n, length in enumerate(_lengths(c)):
        dh[at + length - 1] += s["dht"][n]
        for t in range(at + length - 1, at, -1):
            torch.addcmul(dh[t - 1], a[t], dh[t], out=dh[t - 1])
        part = slice(at, at + length)
        dg[part] = a[part] * dh[part] * torch.cat([s["h0"][n:n + 1].double(), y[at:at + length - 1]])
        dh0.append(a[at] * dh[at])
        at += length
    dx, dbeta = dh, None
    if c["beta"]:
        x = (_exact_held(s["x8"]) if c["bits8"] else s["x"].double()).reshape(-1, D)
        dx, dbeta = dh * s["beta"].double().reshape(-1, D), (dh * x).view(shape)
    return dx.view(shape), dg.view(shape), dbeta, torch.stack(dh0)


def exact_cache(s, c):
    out = s["back"].double()
    for i, j in zip(s["from"].tolist(), s["to"].tolist()):
        out[j] = _exact_round(s["pool"][i].reshape(-1), 127 if c["bits"] == 8 else 7).view(out[j].shape)
    return out


def _exact_norm(x, z, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w * torch.nn.functional.silu(z)


def _exact_norm_grads(x, z, w, dy):
    x, z, w = (t.clone().requires_grad_() for t in (x, z, w))
    _exact_norm(x, z, w).backward(dy)
    return x.grad, z.grad, w.grad


def exact_norm_step(s, c):
    x, z, w, dy = (s[n].double() for n in ("x", "z", "weight", "dy"))
    return _exact_norm(x, z, w), *_exact_norm_grads(_exact_round(x, 127), _exact_round(z, 127), w, dy)


def exact_norm_bwd(s, c):
    return _exact_norm_grads(_exact_held(s["x8"]), _exact_held(s["z8"]), s["weight"].double(), s["dy"].double())


EXACT = {"rec": exact_rec, "rec_steps": exact_rec_steps, "rec_bwd": exact_rec_bwd, "cache": exact_cache,
         "norm_step": exact_norm_step, "norm_bwd": exact_norm_bwd}
