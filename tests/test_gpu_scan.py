"""GPU parity of the gated linear recurrence (over sequences, over a few tokens,
backward) with the float64 definitions in oracle/scan.py.

Bars, from the arithmetic: an output x of magnitude m (the oracle's: the sum of the
absolute values that an fp32 evaluation adds, each with the decay it has had) is
off by at most

    c 2^-24 m + half (|x| + c 2^-24 m),    half = eps/2 of the output's type,

with c the roundings a token brings: 1.5 for e^g (measured against float64 over
its range: 1.47 2^-24 of its value), 1 for the product of decays that carries a
state over a tile, 1 for the sum, 1 for beta x, and under 1 for joining tiles (two
roundings in every 4 tokens or more): 5.  The gradients' products add 3: 8.
"""
import sys

import numpy as np
import pytest
import torch

from oracle import scan as orc

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -24
KINDS = pytest.mark.parametrize("dtype,gate", [(BF, F32), (BF, BF), (F32, F32)], ids=["bf16_fp32", "bf16", "fp32"])


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(name, got, ref, mag, c):
    half = torch.finfo(got.dtype).eps / 2
    tol = c * ULP * mag + half * (np.abs(ref) + c * ULP * mag) + 1e-36
    g = _np(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{name}: not finite"
    over = np.abs(g - ref) / tol
    worst = float(over.max()) if over.size else 0.0
    _say(f"    {name}: worst error {worst:.2f} of the bar")
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bar at {np.unravel_index(over.argmax(), over.shape)}"


CASES = {   # lengths (a tuple: equal), D, beta, initial state, extra columns of the rows
    "plain": ((40, 40), 64, True, False, 0),
    "one_token": ((1,) * 5, 136, False, True, 0),
    "one_channel": ((9, 9, 9), 1, True, True, 2),
    "three_channels": ([5, 130], 3, True, True, 1),
    "odd": ([17, 2, 70], 1001, True, True, 3),
    "packed": ([1, 0, 3, 130, 2, 64, 0, 0, 1, 5, 0], 72, True, True, 8),
    "empty_ends": ([0, 0, 300, 0, 257, 0], 40, False, True, 0),
    "many": ([i % 4 for i in range(600)], 40, True, True, 0),
    "long": ((2100,), 260, True, True, 4),
    "long_rows": ((1025, 1025, 1025), 7, False, False, 0),
    "border_rows": ((256,) * 5, 257, True, True, 0),
    "long_packed": ([3, 900, 0, 2500, 1, 64, 511], 18, True, True, 2),
    "wide": ((33,), 5000, True, False, 0),
    # states handed on over several blocks of 64 tiles
    "blocks": ((36000,), 5, True, True, 0),
    "blocks_rows": ((17500, 17500), 64, False, True, 0),
    "blocks_packed": ([40, 17000, 1, 0, 9000, 9000], 66, True, True, 2),
    "sixty_five": ([300, 700], 65, True, True, 0),
    "sixteen": ([5, 1, 900, 33], 16, True, True, 0),
    "two_channels": ((700, 700), 2, True, True, 1),
    "four_channels": ([1, 2, 700], 4, False, True, 0),
}


def _inputs(name, dtype, gate, seed=7):
    lens, D, with_beta, initial, extra = CASES[name]
    gen, N = torch.Generator().manual_seed(seed + D), len(lens)
    B, T = (1, sum(lens)) if isinstance(lens, list) else (N, lens[0])
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen)  # noqa: E731
    rate = torch.exp(rand(D) * 7 - 6)                # channels that remember two tokens, and hundreds
    g = torch.empty(B, T, D + extra)
    g[..., :D] = -rate * torch.nn.functional.softplus(randn(B, T, D))
    g[..., :D][rand(B, T, D) < 0.02] = -1e30         # some tokens forget everything
    g[..., D:] = 5.0
    x, b = randn(B, T, D + extra).to(dtype), rand(B, T, D + extra).to(gate)
    return {"x": x.to(DEV)[..., extra:], "g": g.to(gate).to(DEV)[..., :D],
            "beta": b.to(DEV)[..., extra:] if with_beta else None,
            "h0": randn(N, D).to(DEV) if initial else None, "dht": randn(N, D).to(DEV) if initial else None,
            "dy": randn(B, T, D).to(dtype).to(DEV),
            "cu": torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=DEV) if isinstance(lens, list) else None,
            "gen": gen}


@KINDS
@pytest.mark.parametrize("name", list(CASES))
def test_recurrence_matches_the_definition(name, dtype, gate):
    gdn = _gdn()
    x = _inputs(name, dtype, gate)
    _say(f"[recurrence] {name} {dtype} {gate}")
    ref, fin, mag, mfin = orc.scan(x["x"], x["g"], x["beta"], x["h0"], x["cu"])
    args = (x["x"], x["g"], x["beta"])
    y, final = gdn.gated_linear_recurrence(*args, initial_state=x["h0"], cu_seqlens=x["cu"])
    torch.cuda.synchronize()
    assert y.dtype == dtype and y.is_contiguous() and final.dtype == F32
    _near("y", y, ref, mag, 5)
    _near("final", final, fin, mfin, 5)
    # no final state; the given buffers; the initial state's buffer updated in place; the same bits again
    out, ws = torch.empty_like(y), torch.full((1 << 23,), 255, dtype=torch.uint8, device=DEV)
    y2, none = gdn.gated_linear_recurrence(*args, initial_state=x["h0"], cu_seqlens=x["cu"], output_final_state=False,
                                           out=out, workspace=ws)
    assert none is None and y2 is out and torch.equal(y2, y)
    if x["h0"] is not None:
        h = x["h0"].clone()
        y3, f3 = gdn.gated_linear_recurrence(*args, initial_state=h, final_state=h, cu_seqlens=x["cu"], workspace=ws)
        assert f3 is h and torch.equal(h, final) and torch.equal(y3, y)


@KINDS
@pytest.mark.parametrize("name", list(CASES))
def test_recurrence_backward_matches_the_definition(name, dtype, gate):
    gdn = _gdn()
    x = _inputs(name, dtype, gate)
    _say(f"[recurrence backward] {name} {dtype} {gate}")
    y, _ = gdn.gated_linear_recurrence(x["x"], x["g"], x["beta"], initial_state=x["h0"], cu_seqlens=x["cu"])
    ref = orc.scan_bwd(x["x"], x["g"], y, x["dy"], x["beta"], x["dht"], x["h0"], x["cu"])
    call = lambda **kw: gdn.gated_linear_recurrence_bwd(  # noqa: E731
        x["x"], x["g"], y, x["dy"], x["beta"], dht=x["dht"], initial_state=x["h0"], cu_seqlens=x["cu"],
        output_dinitial=x["h0"] is not None, **kw)
    got = call()
    torch.cuda.synchronize()
    dx, dg, dbeta, dinitial = got
    assert dx.dtype == dtype and dg.dtype == gate and (dbeta is None) == (x["beta"] is None)
    _near("dx", dx, *ref["dx"], 8)
    _near("dg", dg, *ref["dg"], 8)
    if dbeta is not None:
        assert dbeta.dtype == gate
        _near("dbeta", dbeta, *ref["dbeta"], 8)
    if dinitial is not None:
        _near("dinitial", dinitial, *ref["dinitial"], 8)
    again = call(workspace=torch.full((1 << 23,), 255, dtype=torch.uint8, device=DEV))
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("name", ["plain", "odd", "packed", "long", "three_channels", "one_channel", "long_packed"])
@KINDS
def test_recurrence_backward_from_checkpoints(name, dtype, gate):
    """Gradients at the values that the checkpoints of x and y stand for: the bits of the call on those values."""
    gdn = _gdn()
    x = _inputs(name, dtype, gate)
    y, _ = gdn.gated_linear_recurrence(x["x"], x["g"], x["beta"], initial_state=x["h0"], cu_seqlens=x["cu"])
    x8, y8 = gdn.checkpoint_activation(x["x"]), gdn.checkpoint_activation(y)
    xr, yr = (torch.from_numpy(orc.restore(*c)) for c in (x8, y8))
    _say(f"[recurrence backward, 8 bits] {name} {dtype} {gate}")
    ref = orc.scan_bwd(xr, x["g"], yr, x["dy"], x["beta"], x["dht"], x["h0"], x["cu"])
    with_x = x8 if x["beta"] is not None else None
    call = lambda: gdn.gated_linear_recurrence_bwd(  # noqa: E731
        with_x, x["g"], y8, x["dy"], x["beta"], dht=x["dht"], initial_state=x["h0"], cu_seqlens=x["cu"], output_dinitial=True)
    got = call()
    for t, k in zip(got, ("dx", "dg", "dbeta", "dinitial")):
        if t is not None:
            _near(k, t, *ref[k], 8)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, call()))


@pytest.mark.parametrize("pdt", [F32, BF], ids=["pool_fp32", "pool_bf16"])
@pytest.mark.parametrize("name", ["packed", "odd", "long_packed"])
def test_recurrence_pool(name, pdt):
    gdn = _gdn()
    x = _inputs(name, BF, F32)
    N, D = x["h0"].shape
    P = N + 4
    pool0 = torch.randn(P, D, generator=x["gen"]).to(pdt).to(DEV)
    idx = torch.randperm(P, generator=x["gen"])[:N].to(torch.int32)
    idx[1], idx[2] = -1, P
    ok = (idx >= 0) & (idx < P)
    for read in (True, False):
        start = torch.zeros(N, D, device=DEV)
        if read:
            start[ok] = pool0[idx[ok].long()].float()
        want, fin = gdn.gated_linear_recurrence(x["x"], x["g"], x["beta"], initial_state=start, cu_seqlens=x["cu"])
        pool = pool0.clone()
        y, none = gdn.gated_linear_recurrence(x["x"], x["g"], x["beta"], cu_seqlens=x["cu"], state_pool=pool,
                                              state_indices=idx.to(DEV), read_initial_state=read)
        expect = pool0.clone()
        expect[idx[ok].long()] = fin[ok].to(pdt)
        assert none is None and torch.equal(y, want) and torch.equal(pool, expect)


STEPS = {   # lengths, D, columns, beta, extra
    "decode": ((1,) * 9, 512, 1, False, 0),
    "drafts": ((4,) * 5, 1000, 4, True, 24),
    "ragged": ([2, 0, 5, 1, 3], 515, 3, True, 1),
    "long": ([19, 40], 16, 2, True, 0),
    "few_channels": ((3, 3, 3, 3), 3, 2, True, 0),
    "five_channels": ((2,) * 70, 5, 1, True, 2),
    "last_vector": ((1,) * 21, 1043, 2, False, 0),
    "wide": ((2, 2, 2, 2), 8192, 1, True, 0),
}


@pytest.mark.parametrize("pdt", [F32, BF], ids=["pool_fp32", "pool_bf16"])
@KINDS
@pytest.mark.parametrize("name", list(STEPS))
def test_recurrence_steps_match_the_definition(name, dtype, gate, pdt):
    gdn = _gdn()
    lens, D, cols, with_beta, extra = STEPS[name]
    gen, N = torch.Generator().manual_seed(D), len(lens)
    B, T = (1, sum(lens)) if isinstance(lens, list) else (N, lens[0])
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    xs = randn(B, T, D + extra).to(dtype).to(DEV)[..., extra:]
    g = (-torch.nn.functional.softplus(randn(B, T, D + extra)) * 0.3).to(gate).to(DEV)[..., :D]
    beta = torch.rand(B, T, D, generator=gen).to(gate).to(DEV) if with_beta else None
    P = N * cols + 3
    pool = randn(P, D).to(pdt).to(DEV)
    idx = torch.randperm(P, generator=gen)[:N * cols].to(torch.int32).view(N, cols)
    acc = torch.randint(0, cols + 2, (N,), generator=gen, dtype=torch.int32)
    if N > 3:
        idx[1] = -1
        idx[3, cols - 1] = P
    cu = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=DEV) if isinstance(lens, list) else None
    ref, after, mag, mafter = orc.scan_steps(xs, g, pool, idx, beta, acc, cu)
    _say(f"[recurrence steps] {name} {dtype} {gate} {pdt}")
    pool0 = pool.clone()
    y = gdn.gated_linear_recurrence_steps(xs, g, pool, idx.to(DEV), beta=beta, cu_seqlens=cu, num_accepted=acc.to(DEV))
    torch.cuda.synchronize()
    _near("y", y, ref, mag, 5)
    _near("pool", pool, after, mafter, 5)
    assert torch.equal(pool[mafter.sum(-1) == 0], pool0[mafter.sum(-1) == 0])
    if name == "decode":   # [N, D] rows and [N] indices
        a, b = pool0.clone(), pool0.clone()
        out = torch.empty(N, D, dtype=dtype, device=DEV)
        one = gdn.gated_linear_recurrence_steps(xs[:, 0], g[:, 0], a, idx[:, 0].to(DEV), out=out)
        two = gdn.gated_linear_recurrence_steps(xs, g, b, idx.to(DEV))
        assert one.data_ptr() == out.data_ptr() and one.shape == (N, D)
        assert torch.equal(out, two[:, 0]) and torch.equal(a, b)
