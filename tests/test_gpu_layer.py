"""GPU parity of the operators around the delta rule (recurrent steps, short
convolution, RMS norms, forward and backward) with the float64 definitions in
oracle/layer.py.

Bars, from the arithmetic: the kernels compute in fp32 and round each output
once, so an output x of magnitude m (the oracle's: the sum of the absolute
values that an fp32 evaluation adds, times 1 + |a| where e^-a is formed, whose
argument's rounding grows with a) is off by at most

    c 2^-24 m + half (|x| + c 2^-24 m),    half = eps/2 of the output's type,

with c the number of roundings on the longest path:
  conv 8 (W <= 4 products, the bias, exp, reciprocal, product; the 1.1 bound of
  silu' is in m); its gradients 16, weights' 16 + 112 for the sums (64 tokens of a
  strip, 4 strips, then at most 64 tests' rows and a tree of 6);
  norms 64 (a lane adds at most 16 squares, the group 10 more, then the mean, the
  square root and the products), their gradients 128, weights' 256 (the rows of a
  group and the sums over groups and workgroups);
  steps, as a matrix norm: ||error|| <= 64 2^-24 (the oracle's bound: summed over
  the tokens, whose map is a contraction), 24 for an inner product over K = 128
  in sixteen steps and a tree, the rest for the gates (1.1e-6 of g, and |g| e^g < 0.4).
Histories and untouched slots are equal bit for bit.
"""
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -24
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(name, got, ref, mag, c, dtype=None):
    half = torch.finfo(dtype or got.dtype).eps / 2
    tol = c * ULP * mag + half * (np.abs(ref) + c * ULP * mag) + 1e-36
    g = _np(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{name}: not finite"
    over = np.abs(g - ref) / tol
    worst = float(over.max()) if over.size else 0.0
    _say(f"    {name}: worst error {worst:.2f} of the bar")
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bar at {np.unravel_index(over.argmax(), over.shape)}"


class Draw:
    def __init__(self, seed):
        self.gen = torch.Generator().manual_seed(seed)

    def randn(self, *shape, std=1.0, dtype=F32):
        return (torch.randn(*shape, generator=self.gen) * std).to(dtype)

    def rand(self, *shape):
        return torch.rand(*shape, generator=self.gen)

    def slots(self, P, n):
        return torch.randperm(P, generator=self.gen)[:n].to(torch.int32)


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)


# ---------------------------------------------------------------------------
# Recurrent steps
# ---------------------------------------------------------------------------
STEPS = {   # H, HV, K, V, lengths (an int: equal), columns, raw gates, pool type, L2 norm
    "one_token": (2, 4, 128, 128, (1, 1), 1, False, F32, True),
    "verify": (2, 4, 128, 128, (4, 4, 4), 4, True, F32, True),
    "ragged_bf16": (1, 3, 128, 64, [3, 0, 1, 9, 2], 3, False, BF, True),
    "long": (1, 2, 64, 128, [70, 1], 2, True, F32, True),
    "no_norm": (1, 2, 64, 64, [5, 2, 4], 1, False, BF, False),
    "heads": (4, 4, 64, 64, (2,) * 33, 2, True, F32, True),
    # more columns than lanes, slots behind the 64th read and written
    "many_columns": (1, 1, 64, 64, (69,) * 4, 70, False, F32, True),
    # 256 heads and more, 2048 and more: wider column splits
    "many_heads": (2, 8, 128, 128, [i % 5 for i in range(35)], 2, True, F32, True),
    "many_heads_bf16": (8, 8, 64, 128, (10,) * 33, 1, False, BF, True),
    "wide": (8, 16, 128, 64, [i % 3 for i in range(131)], 1, True, BF, True),
    "wide_rows": (16, 16, 64, 128, (2,) * 129, 1, False, BF, True),
}


def _steps_inputs(name, dtype, seed=11):
    H, HV, K, V, lens, cols, raw, pdt, l2 = STEPS[name]
    d, N, T = Draw(seed), len(lens), sum(lens)
    B, Tr = (1, T) if isinstance(lens, list) else (N, lens[0])
    x = {"q": d.randn(B, Tr, H, K, std=1 if l2 else K ** -0.5, dtype=dtype),
         "k": d.randn(B, Tr, H, K, std=1 if l2 else K ** -0.5, dtype=dtype), "v": d.randn(B, Tr, HV, V, dtype=dtype)}
    P = N * cols + 3
    idx = d.slots(P, N * cols).view(N, cols)
    if N > 2:
        idx[1] = -1                                       # a padding row
        idx[2, 0] = P + 5 if cols > 1 else idx[2, 0]      # a slot outside the pool
    acc = torch.randint(1, cols + 1, (N,), generator=d.gen, dtype=torch.int32)
    if N > 2 and cols > 1:
        acc[2] = cols
    x.update(A_log=d.rand(HV) * 2, dt_bias=d.rand(HV), a=d.randn(B, Tr, HV, dtype=dtype), b=d.randn(B, Tr, HV, dtype=dtype),
             pool=d.randn(P, HV, K, V, std=0.3, dtype=pdt), idx=idx, acc=acc, cu=_cu(lens) if isinstance(lens, list) else None)
    x["g"], x["beta"] = (torch.from_numpy(t) for t in oracle.gating(x["A_log"], x["dt_bias"], x["a"], x["b"]))
    return x


@TYPES
@pytest.mark.parametrize("name", list(STEPS))
def test_steps_match_the_definition(name, dtype):
    gdn = _gdn()
    H, HV, K, V, lens, cols, raw, pdt, l2 = STEPS[name]
    x = _steps_inputs(name, dtype)
    _say(f"[steps] {name} {dtype}")
    if not raw:
        x["g"], x["beta"] = x["g"].float(), x["beta"].float()
    ref, after, bound = layer.steps(x["q"], x["k"], x["v"], x["g"], x["beta"], x["pool"], x["idx"], x["acc"], x["cu"],
                                    use_l2norm=l2)
    dev = {k: None if t is None else t.to(DEV) for k, t in x.items()}
    gates = dict(g=None, beta=None, A_log=dev["A_log"], dt_bias=dev["dt_bias"], a_raw=dev["a"], b_raw=dev["b"]) if raw \
        else dict(g=dev["g"], beta=dev["beta"])
    out = gdn.fused_recurrent_gated_delta_rule_steps(dev["q"], dev["k"], dev["v"], state_pool=dev["pool"],
                                                     state_indices=dev["idx"], cu_seqlens=dev["cu"],
                                                     num_accepted=dev["acc"], use_qk_l2norm_in_kernel=l2, **gates)
    torch.cuda.synchronize()
    assert out.dtype == dtype and out.shape == x["v"].shape
    o, ref = _np(out).reshape(-1, HV, V), ref.reshape(-1, HV, V)
    qn = np.ones((o.shape[0], HV)) if l2 else np.linalg.norm(_np(x["q"]).reshape(-1, H, K), axis=-1).repeat(HV // H, 1)
    seq = np.concatenate([np.full(t1 - t0, n) for n, (t0, t1) in enumerate(layer.ranges(*x["q"].shape[:2], x["cu"]))])
    err = np.linalg.norm(o - ref, axis=-1)
    tol = K ** -0.5 * qn * 128 * ULP * bound[seq] + torch.finfo(dtype).eps / 2 * 1.01 * np.linalg.norm(ref, axis=-1) + 1e-30
    _say(f"    out: worst error {float((err / tol).max()):.2f} of the bar")
    assert (err <= tol).all()
    got = _np(dev["pool"])
    before = _np(x["pool"])
    changed = (after != before).reshape(len(after), -1).any(1)
    for s in range(len(after)):
        if not changed[s]:
            assert (got[s] == before[s]).all(), f"slot {s} was written"
    idx = x["idx"].numpy()
    worst = 0.0
    for n in range(len(idx)):
        for c in range(cols):
            s = idx[n, c]
            if 0 <= s < len(after) and changed[s]:
                e = np.linalg.norm((got[s] - after[s]).reshape(HV, -1), axis=-1)
                t = 64 * ULP * bound[n] + (2.0 ** -8 * 1.01 * np.linalg.norm(after[s].reshape(HV, -1), axis=-1) if pdt == BF else 0)
                worst = max(worst, float((e / t).max()))
    _say(f"    states: worst error {worst:.2f} of the bar")
    assert worst <= 1.0


def test_steps_equal_single_token_decode_and_repeat():
    """Four tokens in one call leave what four one-token calls leave, up to
    rounding, and the same call on the same states gives the same bits."""
    gdn = _gdn()
    x = {k: None if t is None else t.to(DEV) for k, t in _steps_inputs("verify", BF).items()}
    idx = x["idx"][:, :1].contiguous()
    g, beta = x["g"].float(), x["beta"].float()
    pools = []
    for _ in range(2):
        pool = x["pool"].clone()
        o = gdn.fused_recurrent_gated_delta_rule_steps(x["q"], x["k"], x["v"], g, beta, pool, idx, use_qk_l2norm_in_kernel=True)
        pools.append((o, pool))
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    pool = x["pool"].clone()
    for t in range(4):
        one = [x[n][:, t:t + 1].contiguous() for n in "qkv"] + [g[:, t], beta[:, t]]
        o = gdn.fused_recurrent_gated_delta_rule_update(*one, pool, idx[:, 0].contiguous(), use_qk_l2norm_in_kernel=True)
        torch.testing.assert_close(pools[0][0][:, t:t + 1], o, rtol=2.0 ** -7, atol=1e-6)
    torch.testing.assert_close(pools[0][1], pool, rtol=0, atol=1e-5)


def test_steps_slot_beyond_32_bits():
    """A pool of more than 2^31 elements: the last slot's state is read and written."""
    gdn = _gdn()
    HV, K, V = 32, 128, 128
    P = (1 << 31) // (HV * K * V) + 2
    d = Draw(5)
    q, k = (d.randn(1, 2, HV, K, dtype=BF).to(DEV) for _ in range(2))
    v = d.randn(1, 2, HV, V, dtype=BF).to(DEV)
    g, beta = -d.rand(1, 2, HV).to(DEV), d.rand(1, 2, HV).to(DEV)
    small = d.randn(1, HV, K, V, dtype=BF).to(DEV)
    pool = torch.zeros(P, HV, K, V, dtype=BF, device=DEV)
    pool[P - 1] = small[0]
    idx = torch.tensor([P - 1], dtype=torch.int32, device=DEV)
    o = gdn.fused_recurrent_gated_delta_rule_steps(q, k, v, g, beta, pool, idx, use_qk_l2norm_in_kernel=True)
    o2 = gdn.fused_recurrent_gated_delta_rule_steps(q, k, v, g, beta, small, idx * 0, use_qk_l2norm_in_kernel=True)
    assert torch.equal(o, o2) and torch.equal(pool[P - 1], small[0]) and not pool[:P - 1].any()


# ---------------------------------------------------------------------------
# Short convolution
# ---------------------------------------------------------------------------
CONV = {   # lengths (a tuple: equal), D, W, bias, initial, split, extra columns of x's rows, SiLU
    "plain": ((40, 40), 64, 4, False, False, None, 0, True),
    "split_slice": ((37,), 576, 4, True, True, (160, 160, 256), 128, True),
    "packed": ([1, 0, 3, 130, 2, 64, 0, 1, 5], 72, 4, True, True, (24, 24, 24), 0, True),
    "odd": ([17, 2, 70], 1001, 3, True, True, (333, 0, 668), 3, True),
    "one_column": ((9, 9, 9), 1, 2, False, True, None, 2, True),
    "no_silu": ([33, 31], 520, 2, True, False, (8, 512), 0, False),
    "many": ([i % 4 for i in range(300)], 40, 4, False, True, None, 0, True),
    "one_token": ((1,) * 5, 136, 4, True, True, None, 0, True),
    # pieces that end one to three columns into a wave, pieces of fewer columns than a lane's
    "wave_border": ([1, 0, 2, 40, 1, 1], 779, 4, True, True, (515, 5, 259), 0, True),
    "few_columns": ((2, 2, 2), 13, 3, False, True, (7, 3, 3), 1, True),
    "last_parts": ([3, 1, 70, 2], 1043, 4, False, True, (521, 9, 513), 5, True),
}


def _conv_inputs(name, dtype, wdtype=None, seed=23):
    lens, D, W, bias, initial, split, extra, silu = CONV[name]
    d, N = Draw(seed), len(lens)
    B, T = (1, sum(lens)) if isinstance(lens, list) else (N, lens[0])
    wide = d.randn(B, T, D + extra, dtype=dtype).to(DEV)
    return {"x": wide[..., extra:], "w": d.randn(D, W, std=0.5, dtype=wdtype or dtype).to(DEV),
            "b": d.randn(D, std=0.2, dtype=wdtype or dtype).to(DEV) if bias else None,
            "h0": d.randn(N, D, W - 1, dtype=dtype).to(DEV) if initial else None,
            "cu": _cu(lens).to(DEV) if isinstance(lens, list) else None,
            "dy": d.randn(B, T, D, dtype=dtype).to(DEV), "act": "silu" if silu else None, "split": split, "draw": d}


@TYPES
@pytest.mark.parametrize("name", list(CONV))
def test_conv_matches_the_definition(name, dtype):
    gdn = _gdn()
    x = _conv_inputs(name, dtype, F32 if name == "packed" else None)
    _say(f"[conv] {name} {dtype}")
    ref, fin, mag = layer.conv(x["x"], x["w"], x["b"], x["h0"], x["cu"], silu=x["act"] is not None)
    y, final = gdn.causal_conv1d(x["x"], x["w"], x["b"], initial_state=x["h0"], cu_seqlens=x["cu"], activation=x["act"],
                                 split_sizes=x["split"])
    torch.cuda.synchronize()
    if x["split"]:
        assert [t.shape[-1] for t in y] == list(x["split"]) and all(t.is_contiguous() for t in y)
        y = torch.cat(y, -1)
    _near("y", y, ref, mag, 8)
    assert final.dtype == dtype and (_np(final) == fin).all()
    # no final state; the initial state's buffer updated in place
    y2, none = gdn.causal_conv1d(x["x"], x["w"], x["b"], initial_state=x["h0"], cu_seqlens=x["cu"], activation=x["act"],
                                 output_final_state=False)
    assert none is None and torch.equal(y2, y)
    if x["h0"] is not None:
        h = x["h0"].clone()
        y3, f3 = gdn.causal_conv1d(x["x"], x["w"], x["b"], initial_state=h, final_state=h, cu_seqlens=x["cu"],
                                   activation=x["act"])
        assert f3 is h and torch.equal(h, final) and torch.equal(y3, y)


@TYPES
def test_conv_pool(dtype):
    gdn = _gdn()
    x = _conv_inputs("packed", dtype)
    N, D, W1 = x["h0"].shape
    P = N + 4
    pool0 = x["draw"].randn(P, D, W1, dtype=dtype).to(DEV)
    idx = x["draw"].slots(P, N)
    idx[3], idx[4] = -1, P
    for read in (True, False):
        start = torch.zeros_like(x["h0"])
        ok = (idx >= 0) & (idx < P)
        if read:
            start[ok] = pool0[idx[ok].long()]
        want, fin = gdn.causal_conv1d(x["x"], x["w"], x["b"], initial_state=start, cu_seqlens=x["cu"])
        pool = pool0.clone()
        y, none = gdn.causal_conv1d(x["x"], x["w"], x["b"], cu_seqlens=x["cu"], conv_state_pool=pool,
                                    conv_state_indices=idx.to(DEV), read_initial_state=read)
        expect = pool0.clone()
        expect[idx[ok].long()] = fin[ok]
        assert none is None and torch.equal(y, want) and torch.equal(pool, expect)


UPDATE = {   # lengths, D, W, columns, bias, split, extra
    "decode": ((1,) * 9, 512, 4, 1, False, (128, 128, 256), 0),
    "drafts": ((4,) * 5, 1000, 4, 4, True, None, 24),
    "ragged": ([2, 0, 5, 1, 3], 515, 3, 3, True, (100, 200, 215), 1),
    "long": ([19, 40], 16, 2, 1, False, None, 0),
    "wave_border": ((1,) * 40, 518, 4, 1, True, (259, 3, 256), 0),
    "last_parts": ((3,) * 21, 1043, 4, 2, False, (517, 9, 517), 3),
}


@TYPES
@pytest.mark.parametrize("name", list(UPDATE))
def test_conv_update_matches_the_definition(name, dtype):
    gdn = _gdn()
    lens, D, W, cols, bias, split, extra = UPDATE[name]
    d, N = Draw(31), len(lens)
    B, T = (1, sum(lens)) if isinstance(lens, list) else (N, lens[0])
    wide = d.randn(B, T, D + extra, dtype=dtype).to(DEV)
    xs, w = wide[..., :D], d.randn(D, W, std=0.5, dtype=dtype).to(DEV)
    b = d.randn(D, std=0.2, dtype=dtype).to(DEV) if bias else None
    P = N * cols + 3
    pool = d.randn(P, D, W - 1, dtype=dtype).to(DEV)
    idx = d.slots(P, N * cols).view(N, cols)
    acc = torch.randint(0, cols + 2, (N,), generator=d.gen, dtype=torch.int32)
    if N > 3:
        idx[1] = -1
        idx[3, cols - 1] = P
    cu = _cu(lens).to(DEV) if isinstance(lens, list) else None
    ref, after, mag = layer.conv_update(xs, w, pool, idx, b, acc, cu)
    _say(f"[conv update] {name} {dtype}")
    y = gdn.causal_conv1d_update(xs, w, pool, idx.to(DEV), b, cu_seqlens=cu, num_accepted=acc.to(DEV), split_sizes=split)
    torch.cuda.synchronize()
    _near("y", torch.cat(y, -1) if split else y, ref, mag, 8)
    assert (_np(pool) == after).all()
    if name == "decode":   # [N, D] rows and [N] indices
        pool2 = d.randn(P, D, W - 1, dtype=dtype).to(DEV)
        a = gdn.causal_conv1d_update(xs[:, 0], w, pool2.clone(), idx[:, 0].to(DEV), b)
        c = gdn.causal_conv1d_update(xs, w, pool2, idx.to(DEV), b)
        assert a.shape == (N, D) and torch.equal(a, c[:, 0])


@TYPES
@pytest.mark.parametrize("name", list(CONV))
def test_conv_backward_matches_the_definition(name, dtype):
    gdn = _gdn()
    x = _conv_inputs(name, dtype, F32 if name == "odd" else None)
    _say(f"[conv backward] {name} {dtype}")
    ref = layer.conv_bwd(x["x"], x["w"], x["dy"], x["b"], x["h0"], x["cu"], silu=x["act"] is not None)
    dy = [t.contiguous() for t in x["dy"].split(x["split"], -1)] if x["split"] else x["dy"]
    call = lambda: gdn.causal_conv1d_bwd(x["x"], x["w"], dy, x["b"], initial_state=x["h0"], cu_seqlens=x["cu"],
                                         activation=x["act"], output_dinitial=x["h0"] is not None)
    dx, dw, db, dh = call()
    torch.cuda.synchronize()
    assert dx.dtype == dtype and dw.dtype == F32 and (db is None) == (x["b"] is None)
    _near("dx", dx, *ref["dx"], 16)
    _near("dweight", dw, *ref["dweight"], 128)
    if db is not None:
        _near("dbias", db, *ref["dbias"], 128)
    if dh is not None:
        _near("dinitial", dh, *ref["dinitial"], 16)
    again = call()
    assert all(a is b is None or torch.equal(a, b) for a, b in zip((dx, dw, db, dh), again))


# ---------------------------------------------------------------------------
# RMS norms
# ---------------------------------------------------------------------------
@TYPES
@pytest.mark.parametrize("lead,D", [((5, 4), 128), ((3, 1, 6), 64), ((7,), 1), ((2, 3), 100), ((9, 2), 129), ((3,), 512),
                                    ((2, 2), 777), ((2,), 1024), ((300, 32), 128), ((3, 5), 1021), ((700, 9), 5),
                                    ((900, 10), 187), ((257, 9), 252), ((70, 3), 9), ((5, 2), 15)])
def test_gated_norm_and_backward(lead, D, dtype):
    gdn = _gdn()
    d = Draw(D)
    x, dy, w = d.randn(*lead, D, dtype=dtype), d.randn(*lead, D, dtype=dtype), (d.randn(D, std=0.3) + 1).to(dtype)
    heads = lead[-1] if len(lead) > 1 else 1
    wide = d.randn(*lead[:-1] if heads > 1 else lead, heads * D + 5, std=2.0, dtype=dtype)
    z = wide[..., 5:].view(*lead, D) if heads > 1 or len(lead) == 1 else wide[..., 5:].reshape(*lead, D)
    _say(f"[gated norm] {lead} {D} {dtype}")
    ref, mag = layer.gated_norm(x, z, w)
    xd, dyd, wd = x.to(DEV), dy.to(DEV), w.to(DEV)
    zd = wide.to(DEV)[..., 5:].view(*lead, D)
    _near("y", gdn.fused_gated_rms_norm(xd, zd, wd), ref, mag, 64)
    assert torch.equal(gdn.fused_gated_rms_norm(xd, zd.contiguous(), wd.float()), gdn.fused_gated_rms_norm(xd, zd, wd))
    got = gdn.fused_gated_rms_norm_bwd(xd, zd, wd, dyd)
    grads = layer.gated_norm_bwd(x, z, w, dy)
    for t, name, c in zip(got, ("dx", "dz", "dweight"), (128, 128, 256)):
        _near(name, t, *grads[name], c)
    assert all(torch.equal(a, b) for a, b in zip(got, gdn.fused_gated_rms_norm_bwd(xd, zd, wd, dyd)))


@TYPES
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (70, 64), (5, 520), (4, 1025), (3, 2048), (700, 2048), (2, 2500),
                                    (3, 4096), (2, 5121), (2, 8192), (3, 9001), (2, 16384), (2, 16383), (3, 1032),
                                    (900, 1027), (600, 4097), (9000, 3), (400, 10240), (65, 9), (33, 15)])
def test_add_norm_and_backward(rows, D, dtype):
    gdn = _gdn()
    d = Draw(rows + D)
    x, res, dy, dh = (d.randn(rows, D, std=s, dtype=dtype) for s in (1.0, 2.0, 1.0, 1.0))
    w = d.randn(D, std=0.3, dtype=dtype)
    kw = dict(residual_scale=0.7, weight_offset=1.0)
    _say(f"[add norm] {rows} x {D} {dtype}")
    ref, h = layer.add_norm(x, res, w, **kw)
    xd, rd, dyd, dhd, wd = (t.to(DEV) for t in (x, res, dy, dh, w))
    y, hid = gdn.fused_add_rms_norm(xd, rd, wd, **kw)
    # hidden = residual + scale x may cancel (to zero, where the fp32 scale is not 0.7): its error is a share of
    # the terms' size, and y = hidden r (w + 1) has that error times r |w + 1|, whatever hidden is
    size = np.abs(_np(res)) + 0.7 * np.abs(_np(x))
    _near("hidden", hid, h, size, 2)
    _near("y", y, ref, np.abs(ref) + size * np.abs(_np(w) + 1) / np.sqrt((h * h).mean(-1, keepdims=True) + 1e-6), 64)
    inplace = rd.clone()
    y2, h2 = gdn.fused_add_rms_norm(xd, inplace, wd, hidden=inplace, **kw)
    assert h2 is inplace and torch.equal(h2, hid) and torch.equal(y2, y)
    y3, h3 = gdn.fused_add_rms_norm(xd, None, wd)
    ref3, _ = layer.add_norm(x, None, w)
    _near("y without residual", y3, ref3, np.abs(ref3), 64)
    assert torch.equal(h3, xd)
    got = gdn.fused_add_rms_norm_bwd(dyd, dhd, hid, wd, **kw)
    grads = layer.add_norm_bwd(dy, dh, hid, w, **kw)
    for t, name, c in zip(got, ("dx", "dresidual", "dweight"), (128, 128, 256)):
        _near(name, t, *grads[name], c)
    none, dres, dw = gdn.fused_add_rms_norm_bwd(dyd, None, hid, wd, output_dx=False, weight_offset=1.0)
    grads = layer.add_norm_bwd(dy, None, hid, w, weight_offset=1.0)
    assert none is None and torch.equal(dw, got[2])
    _near("dresidual alone", dres, *grads["dresidual"], 128)


def test_inputs_off_alignment():
    """Contiguous tensors that begin one element into their storage: every
    operator takes them and gives the bits of the aligned call."""
    gdn = _gdn()

    def off(t):
        if t is None or t.dtype not in (BF, F32):
            return t
        u = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        return u.copy_(t)
    for dtype in (BF, F32):
        x = {k: None if t is None else t.to(DEV) for k, t in _steps_inputs("verify", dtype).items()}
        g, beta = x["g"].float(), x["beta"].float()
        outs = []
        for f in (lambda t: t, off):
            pool = x["pool"].clone()
            o = gdn.fused_recurrent_gated_delta_rule_steps(f(x["q"]), f(x["k"]), f(x["v"]), f(g), f(beta), pool, x["idx"],
                                                           num_accepted=x["acc"], use_qk_l2norm_in_kernel=True,
                                                           out=f(torch.empty_like(x["v"])))
            outs.append((o, pool))
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        c = _conv_inputs("packed", dtype)
        xs = c["x"].contiguous()
        for call in (lambda f: gdn.causal_conv1d(f(xs), f(c["w"]), f(c["b"]), initial_state=f(c["h0"]), cu_seqlens=c["cu"]),
                     lambda f: gdn.causal_conv1d_bwd(f(xs), f(c["w"]), f(c["dy"]), f(c["b"]), initial_state=f(c["h0"]),
                                                     cu_seqlens=c["cu"], output_dinitial=True),
                     lambda f: gdn.fused_gated_rms_norm_bwd(f(xs), f(c["dy"]), f(c["w"][:, 0].contiguous()), f(c["dy"])),
                     lambda f: gdn.fused_add_rms_norm(f(xs), f(c["dy"]), f(c["w"][:, 0].contiguous()))):
            assert all(torch.equal(a, b) for a, b in zip(call(lambda t: t), call(off)))


def test_padding_rows_and_foreign_slots_do_not_leak():
    """NaN in the inputs of padding rows and in slots that no row names change
    nothing; a slot named for every column of a row ends with its last state."""
    gdn = _gdn()
    x = {k: None if t is None else t.to(DEV) for k, t in _steps_inputs("verify", BF).items()}
    x["idx"][2] = x["idx"][2, 1]
    named = set(i for i in x["idx"].flatten().tolist() if i >= 0)
    foreign = [i for i in range(x["pool"].shape[0]) if i not in named]
    outs = []
    for bad in (False, True):
        q, k, v, a, b, pool = (x[n].clone() for n in ("q", "k", "v", "a", "b", "pool"))
        if bad:
            for t in (q, k, v, a, b):
                t[1] = float("nan")                       # row 1 is padding
            pool[foreign] = float("nan")
        o = gdn.fused_recurrent_gated_delta_rule_steps(q, k, v, None, None, pool, x["idx"], num_accepted=x["acc"],
                                                       use_qk_l2norm_in_kernel=True, A_log=x["A_log"],
                                                       dt_bias=x["dt_bias"], a_raw=a, b_raw=b)
        outs.append((o, pool[sorted(named)]))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and not outs[0][0][1].any()
    one = x["pool"].clone()
    gdn.fused_recurrent_gated_delta_rule_steps(x["q"], x["k"], x["v"], None, None, one, x["idx"][:, 1].contiguous(),
                                               use_qk_l2norm_in_kernel=True, A_log=x["A_log"], dt_bias=x["dt_bias"],
                                               a_raw=x["a"], b_raw=x["b"])
    slot = int(x["idx"][2, 1])
    assert torch.equal(outs[0][1][sorted(named).index(slot)], one[slot])
    d = Draw(6)
    xs, w, pool = d.randn(4, 3, 40, dtype=BF).to(DEV), d.randn(40, 4, dtype=BF).to(DEV), d.randn(9, 40, 3, dtype=BF).to(DEV)
    idx = torch.tensor([[1, 2, 3], [-1, 4, 4], [6, 6, 6], [5, 9, 7]], dtype=torch.int32, device=DEV)
    ref, after, mag = layer.conv_update(xs, w, pool, idx)
    xs[1] = float("nan")
    pool[0] = pool[8] = float("nan")
    y = gdn.causal_conv1d_update(xs, w, pool, idx)
    _near("y", y, ref, mag, 8)
    assert (_np(pool[1:8]) == after[1:8]).all()


def test_two_streams_at_once():
    """The same operators on two streams at once, each call with its own outputs
    and workspace, give what they give alone."""
    gdn = _gdn()
    x = _conv_inputs("split_slice", BF)
    d = Draw(8)
    h, dy = d.randn(3000, 1024, dtype=BF).to(DEV), d.randn(3000, 1024, dtype=BF).to(DEV)
    w = d.randn(1024, dtype=BF).to(DEV)
    dys = [t.contiguous() for t in x["dy"].split(x["split"], -1)]

    def step():
        return [*gdn.fused_add_rms_norm_bwd(dy, None, h, w), *gdn.fused_gated_rms_norm_bwd(h, dy, w, dy),
                *(t for t in gdn.causal_conv1d_bwd(x["x"], x["w"], dys, x["b"], initial_state=x["h0"]) if t is not None)]
    alone = step()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step()
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, alone))


def test_rows_behind_the_last_sequence():
    """A packed batch padded to a fixed T: the rows behind the last sequence stay
    as they were, the others and the weights' gradients are the unpadded call's."""
    gdn = _gdn()
    x = _conv_inputs("packed", BF)
    T, D, pad = x["x"].shape[1], x["x"].shape[2], 41
    more = x["draw"].randn(1, pad, D, dtype=BF).to(DEV).fill_(float("nan"))
    wide, dy = torch.cat([x["x"], more], 1), torch.cat([x["dy"], more], 1)
    out = torch.full_like(wide, 7)
    y, fin = gdn.causal_conv1d(wide, x["w"], x["b"], initial_state=x["h0"], cu_seqlens=x["cu"], out=out)
    want, wfin = gdn.causal_conv1d(x["x"], x["w"], x["b"], initial_state=x["h0"], cu_seqlens=x["cu"])
    assert y is out and torch.equal(y[:, :T], want) and torch.equal(fin, wfin) and (y[:, T:] == 7).all()
    got = gdn.causal_conv1d_bwd(wide, x["w"], dy, x["b"], initial_state=x["h0"], cu_seqlens=x["cu"], output_dinitial=True)
    ref = layer.conv_bwd(x["x"], x["w"], x["dy"], x["b"], x["h0"], x["cu"])
    _near("dx", got[0][:, :T], *ref["dx"], 16)
    _near("dweight", got[1], *ref["dweight"], 128)
    _near("dbias", got[2], *ref["dbias"], 128)
    _near("dinitial", got[3], *ref["dinitial"], 16)
    s = {k: None if t is None else t.to(DEV) for k, t in _steps_inputs("ragged_bf16", BF).items()}
    n = s["v"].shape[1]
    outs = []
    for extra in (0, 9):
        q, k, v, a, b = (torch.cat([s[i], torch.full_like(s[i][:, :1], float("nan")).expand(-1, extra, *s[i].shape[2:])], 1)
                         for i in ("q", "k", "v", "a", "b"))
        pool, out = s["pool"].clone(), torch.full_like(v, 7)
        gdn.fused_recurrent_gated_delta_rule_steps(q, k, v, None, None, pool, s["idx"], cu_seqlens=s["cu"], num_accepted=s["acc"],
                                                   A_log=s["A_log"], dt_bias=s["dt_bias"], a_raw=a, b_raw=b, out=out)
        outs.append((out[:, :n], pool))
        assert (out[:, n:] == 7).all()
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_norm_without_rows():
    gdn = _gdn()
    w = torch.ones(64, device=DEV)
    x = torch.empty(0, 64, device=DEV)
    assert gdn.fused_gated_rms_norm(x, x, w).shape == (0, 64)
    assert gdn.fused_add_rms_norm(x, x, w)[1].shape == (0, 64)
    for dw in (gdn.fused_gated_rms_norm_bwd(x, x, w, x)[2], gdn.fused_add_rms_norm_bwd(x, None, x, w)[2]):
        assert torch.equal(dw, torch.zeros_like(w))


def test_conv_without_tokens():
    gdn = _gdn()
    d = Draw(2)
    w, h = d.randn(24, 4).to(DEV), d.randn(3, 24, 3).to(DEV)
    x = torch.empty(3, 0, 24, device=DEV)
    y, fin = gdn.causal_conv1d(x, w, initial_state=h)
    assert y.shape == (3, 0, 24) and torch.equal(fin, h)
    dx, dw, db, dh = gdn.causal_conv1d_bwd(x, w, x, w[:, 0].contiguous(), initial_state=h, output_dinitial=True)
    assert dx.shape == x.shape and not dw.any() and not db.any() and not dh.any() and dh.shape == h.shape
    pool = h.clone()
    idx = torch.arange(3, dtype=torch.int32, device=DEV)
    assert gdn.causal_conv1d_update(x, w, pool, idx).shape == x.shape and torch.equal(pool, h)


# ---------------------------------------------------------------------------
# Together, as a layer runs them
# ---------------------------------------------------------------------------
def _layer(seed, N, T, dtype=BF):
    H, HV, K, V, hidden = 2, 4, 64, 128, 384
    D = 2 * H * K + HV * V
    d = Draw(seed)
    t = {"x": d.randn(N, T, hidden, dtype=dtype), "res": d.randn(N, T, hidden, dtype=dtype),
         "w_in": d.randn(hidden, std=0.1, dtype=dtype), "proj": d.randn(hidden, D + HV * V + 2 * HV, std=hidden ** -0.5, dtype=dtype),
         "conv": d.randn(D, 4, std=0.5, dtype=dtype), "A_log": d.rand(HV) * 2, "dt_bias": d.rand(HV),
         "w_out": d.randn(V, std=0.1) + 1}
    return (H, HV, K, V, D), {k: v.to(DEV) for k, v in t.items()}


def test_decode_layer_in_a_graph():
    """Residual norm, convolution, recurrent steps and gated norm of a batch of
    drafts, captured in one graph: every replay, with eager work between, equals
    the eager run."""
    gdn = _gdn()
    N, T, cols = 6, 3, 3
    (H, HV, K, V, D), t = _layer(1, N, T)
    P = N * cols + 2
    d = Draw(9)
    idx = d.slots(P, N * cols).view(N, cols)
    idx[4] = -1
    idx, acc = idx.to(DEV), torch.tensor([1, 2, 3, 1, 2, 3], dtype=torch.int32, device=DEV)
    conv0, state0 = d.randn(P, D, 3, dtype=BF).to(DEV), d.randn(P, HV, K, V, std=0.1).to(DEV)
    conv, state, res = conv0.clone(), state0.clone(), t["res"].clone()

    def step():
        y, _ = gdn.fused_add_rms_norm(t["x"], res, t["w_in"], weight_offset=1.0, hidden=res)
        p = (y.float().view(N * T, -1) @ t["proj"].float()).to(BF).view(N, T, -1)
        qkv, z, a, b = p.split((D, HV * V, HV, HV), -1)
        q, k, v = gdn.causal_conv1d_update(qkv, t["conv"], conv, idx, num_accepted=acc, split_sizes=(H * K, H * K, HV * V))
        o = gdn.fused_recurrent_gated_delta_rule_steps(
            q.view(N, T, H, K), k.view(N, T, H, K), v.view(N, T, HV, V), None, None, state, idx, num_accepted=acc,
            use_qk_l2norm_in_kernel=True, A_log=t["A_log"], dt_bias=t["dt_bias"], a_raw=a.contiguous(), b_raw=b.contiguous())
        return gdn.fused_gated_rms_norm(o, z.unflatten(-1, (HV, V)), t["w_out"])

    def reset():
        conv.copy_(conv0), state.copy_(state0), res.copy_(t["res"])

    _say("[layer] decode in a graph")
    eager = [u.clone() for u in (step(), conv, state, res)]
    torch.cuda.synchronize()
    # the pieces agree with the definitions, each fed the eager run's own inputs
    y, h = layer.add_norm(t["x"], t["res"], t["w_in"], weight_offset=1.0)
    _near("hidden", eager[3], h, np.abs(_np(t["x"])) + np.abs(_np(t["res"])), 2)
    assert not eager[0][4].any() and torch.equal(eager[1][P - 1], conv0[P - 1]) == (P - 1 not in idx.cpu().tolist())
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        out.fill_(7)
        reset()
        torch.randn(1 << 20, device=DEV).mul_(2.0).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip((out, conv, state, res), eager):
            assert torch.equal(got, want), f"replay {i}"


@pytest.mark.parametrize("packed", [False, True])
def test_training_layer(packed):
    """Forward and backward of convolution, chunked delta rule and gated norm,
    chained, against the float64 definitions chained the same way."""
    gdn = _gdn()
    N, T = (1, 150) if packed else (2, 70)
    (H, HV, K, V, D), t = _layer(4, N, T, F32)
    d = Draw(12)
    p = d.randn(N, T, D + HV * V).to(DEV)
    qkv, z = p[..., :D], p[..., D:].unflatten(-1, (HV, V))
    g, beta = -d.rand(N, T, HV).to(DEV), d.rand(N, T, HV).to(DEV)
    dy = d.randn(N, T, HV, V).to(DEV)
    cu = torch.tensor([0, 3, 3, 90, 150], dtype=torch.int32, device=DEV) if packed else None
    sizes = (H * K, H * K, HV * V)
    _say(f"[layer] training packed={packed}")
    (q, k, v), _ = gdn.causal_conv1d(qkv, t["conv"], cu_seqlens=cu, split_sizes=sizes)
    q, k, v = q.view(N, T, H, K), k.view(N, T, H, K), v.view(N, T, HV, V)
    o, _ = gdn.chunk_gated_delta_rule(q, k, v, g, beta, cu_seqlens=cu, use_qk_l2norm_in_kernel=True)
    y = gdn.fused_gated_rms_norm(o, z, t["w_out"])
    do, dz, dw = gdn.fused_gated_rms_norm_bwd(o, z, t["w_out"], dy)
    dq, dk, dv, *_ = gdn.chunk_gated_delta_rule_bwd(q, k, v, g, beta, do, cu_seqlens=cu, use_qk_l2norm_in_kernel=True)
    dqkv, dconv, _, _ = gdn.causal_conv1d_bwd(qkv, t["conv"], [u.view(N, T, -1) for u in (dq, dk, dv)], cu_seqlens=cu)
    torch.cuda.synchronize()
    r = layer.conv(qkv, t["conv"], cu_seqlens=cu)[0]
    rq, rk, rv = (r[..., a:b].reshape(N, T, h, -1) for a, b, h in ((0, H * K, H), (H * K, 2 * H * K, H), (2 * H * K, D, HV)))
    ro, _ = oracle.recurrent(*(u.astype(np.float32) for u in (rq, rk, rv)), _np(g).astype(np.float32),
                             _np(beta).astype(np.float32), use_l2norm=True, cu_seqlens=None if cu is None else cu.cpu().numpy())
    ry, _ = layer.gated_norm(ro, z, t["w_out"])
    rg = layer.gated_norm_bwd(ro, z, t["w_out"], dy)
    from oracle.backward import backward
    rb = backward(*(u.astype(np.float32) for u in (rq, rk, rv)), _np(g).astype(np.float32), _np(beta).astype(np.float32),
                  rg["dx"][0], use_l2norm=True, cu_seqlens=None if cu is None else cu.cpu().numpy())
    rdy = np.concatenate([u.reshape(N, T, -1) for u in (rb["dq"], rb["dk"], rb["dv"])], -1)
    rc = layer.conv_bwd(qkv, t["conv"], rdy, cu_seqlens=cu)
    # fp32 through three operators: the delta rule's fp32 bar is 1e-4 of max|ref|; the norm divides by the row's
    # size and the maps around it are linear, so the bar holds with the same factor of ten for the chain
    for name, got, ref in (("y", y, ry), ("dz", dz, rg["dz"][0]), ("dweight", dw, rg["dweight"][0]),
                           ("dqkv", dqkv, rc["dx"][0]), ("dconv", dconv, rc["dweight"][0])):
        err = np.abs(_np(got) - ref).max() / np.abs(ref).max()
        _say(f"    {name}: {err:.1e}")
        assert err <= 1e-3, name


def test_backward_passes_in_a_graph():
    gdn = _gdn()
    x = _conv_inputs("packed", BF)
    d = Draw(3)
    h, dy = d.randn(70, 2048, dtype=BF).to(DEV), d.randn(70, 2048, dtype=BF).to(DEV)
    w = d.randn(2048, dtype=BF).to(DEV)
    o, z, do, wo = (d.randn(33, 4, 128, dtype=BF).to(DEV) for _ in range(4))

    def step():
        return [*gdn.causal_conv1d_bwd(x["x"], x["w"], x["dy"], x["b"], initial_state=x["h0"], cu_seqlens=x["cu"],
                                       output_dinitial=True),
                *gdn.fused_add_rms_norm_bwd(dy, None, h, w, weight_offset=1.0),
                *gdn.fused_gated_rms_norm_bwd(o, z, wo[0, 0].contiguous(), do),
                *gdn.causal_conv1d(x["x"], x["w"], x["b"], initial_state=x["h0"], cu_seqlens=x["cu"])]
    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # and on a stream that is not the tensors' own
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.fill_(7)
        torch.randn(1 << 20, device=DEV).mul_(2.0).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out))
