"""Host-side checks of the operators around the delta rule (no GPU): every
refused argument of the C entry points and of the Python wrappers.  The argument
pointers are never dereferenced: every call fails a check first, or has nothing
to compute."""
import ctypes

import pytest
import torch

import gated_deltanet_chunked_delta_amd as gdn

FAKE = 1 << 20
P = ctypes.c_void_p
BF, F32 = gdn.GDN_BF16, gdn.GDN_F32


def _lib():
    from gated_deltanet_chunked_delta_amd import _binding_layer
    return _binding_layer._load()


def _ref(s):
    return None if s is None else ctypes.byref(s)


# ---------------------------------------------------------------------------
# Recurrent steps
# ---------------------------------------------------------------------------
STEP_SHAPE = dict(B=3, T=4, H=2, HV=4, K=128, V=128, N=3, dtype=BF)


def _steps(shape=None, pool=None, cu=None, no_pool=False, no_shape=False, gates="none", **ptr):
    s = gdn.make_shape(**{**STEP_SHAPE, **(shape or {})})
    pl = gdn.gdn_step_pool(**{**dict(data=FAKE, indices=FAKE, num_accepted=FAKE, pool_size=9, cols=2, dtype=F32), **(pool or {})})
    gt = {"none": None, "raw": gdn.gdn_gates(FAKE, FAKE, FAKE, FAKE), "bad": gdn.gdn_gates(FAKE, FAKE, None, FAKE),
          "off": gdn.gdn_gates(FAKE, FAKE, FAKE + 2, FAKE)}[gates]
    a = {n: ptr.get(n, FAKE) for n in ("q", "k", "v", "g", "beta", "out")}
    return _lib().gdn_recurrent_steps(a["q"], a["k"], a["v"], a["g"], a["beta"], _ref(gt), 1.0, 1,
                                      None if no_pool else ctypes.byref(pl), cu, a["out"],
                                      None if no_shape else ctypes.byref(s), None)


@pytest.mark.parametrize("kw,want", [
    (dict(no_shape=True), -1), (dict(no_pool=True), -1),
    (dict(shape=dict(N=2)), -2), (dict(cu=FAKE), -2),                       # N != B; B != 1 with cu_seqlens
    (dict(shape=dict(B=1, N=0), cu=FAKE), -2),                              # tokens without a sequence
    (dict(shape=dict(T=-1)), -2), (dict(shape=dict(H=1, HV=1 << 23, B=2, N=2)), -2),   # too many workgroups
    (dict(shape=dict(dtype=7)), -3), (dict(pool=dict(dtype=2)), -3),
    (dict(shape=dict(K=96)), -4), (dict(shape=dict(V=32)), -4), (dict(shape=dict(H=3)), -4),
    (dict(q=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(g=None), -1), (dict(beta=None), -1),
    (dict(gates="bad"), -1), (dict(gates="off"), -7),
    (dict(pool=dict(data=None)), -1), (dict(pool=dict(indices=None)), -1),
    (dict(pool=dict(pool_size=0)), -2), (dict(pool=dict(cols=0)), -2),
    (dict(pool=dict(data=FAKE + 8)), -7), (dict(pool=dict(data=FAKE + 4, dtype=BF)), -7),
    (dict(pool=dict(indices=FAKE + 2)), -7), (dict(pool=dict(num_accepted=FAKE + 1)), -7),
    (dict(k=FAKE + 1), -7), (dict(out=FAKE + 1), -7), (dict(g=FAKE + 2), -7),
    (dict(shape=dict(B=1, N=3), cu=FAKE + 2), -7),
    (dict(shape=dict(T=0)), 0), (dict(shape=dict(B=0, N=0)), 0),            # nothing to compute
])
def test_steps_refusals(kw, want):
    assert _steps(**kw) == want


# ---------------------------------------------------------------------------
# Convolution
# ---------------------------------------------------------------------------
def _pieces(dims=(8, 8, 16), ptr=FAKE):
    p = gdn.gdn_conv_pieces()
    for i, n in enumerate(dims):
        p.ptr[i], p.dim[i] = ptr, n
    return p


CONV_SHAPE = dict(B=2, T=5, D=32, W=4, N=2, dtype=BF, weight_dtype=BF, x_stride=32)


def _conv(entry, shape=None, pieces=None, cu=None, no_shape=False, pool=None, no_pool=False, ws=FAKE, ws_bytes=1 << 30, **ptr):
    s = gdn.gdn_conv_shape(**{**CONV_SHAPE, **(shape or {})})
    a = {n: ptr.get(n, FAKE) for n in ("x", "weight", "bias", "initial", "final", "dx", "dweight", "dbias", "dinitial")}
    pc = _ref(_pieces() if pieces is None else pieces if pieces != "none" else None)
    sp = None if no_shape else ctypes.byref(s)
    head = (a["x"], a["weight"], a["bias"], 1)
    if entry == "fwd":
        return _lib().gdn_conv_fwd(*head, a["initial"], cu, pc, a["final"], sp, None)
    if entry == "pool":
        pl = gdn.gdn_state_pool(**{**dict(data=FAKE, indices=FAKE, pool_size=4, dtype=BF, read_initial=1), **(pool or {})})
        return _lib().gdn_conv_fwd_pool(*head, None if no_pool else ctypes.byref(pl), cu, pc, sp, None)
    if entry == "update":
        pl = gdn.gdn_step_pool(**{**dict(data=FAKE, indices=FAKE, num_accepted=None, pool_size=4, cols=1, dtype=BF), **(pool or {})})
        return _lib().gdn_conv_update(*head, None if no_pool else ctypes.byref(pl), cu, pc, sp, None)
    return _lib().gdn_conv_bwd(*head, a["initial"], cu, pc, a["dx"], a["dweight"], a["dbias"], a["dinitial"], sp, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("entry", ["fwd", "pool", "update", "bwd"])
@pytest.mark.parametrize("kw,want", [
    (dict(no_shape=True), -1), (dict(pieces="none"), -1),
    (dict(shape=dict(T=-1)), -2), (dict(shape=dict(N=3)), -2), (dict(cu=FAKE), -2), (dict(shape=dict(D=0)), -2),
    (dict(shape=dict(B=1, N=0), cu=FAKE), -2), (dict(shape=dict(B=1 << 16, N=1 << 16, T=1 << 16)), -2),
    (dict(shape=dict(x_stride=31)), -2), (dict(shape=dict(x_stride=(1 << 31) + 1)), -2),
    (dict(shape=dict(D=(1 << 26) + 1, x_stride=1 << 27)), -2),
    (dict(shape=dict(B=1, T=1 << 28, N=1, D=1 << 14, x_stride=1 << 14), pieces=_pieces((1 << 14, 0, 0))), -2),   # grid
    (dict(shape=dict(dtype=4)), -3), (dict(shape=dict(weight_dtype=-1)), -3),
    (dict(shape=dict(W=1)), -4), (dict(shape=dict(W=5)), -4), (dict(shape=dict(dtype=F32)), -4),   # bf16 weights of fp32 x
    (dict(pieces=_pieces((8, 8, 8))), -2), (dict(pieces=_pieces((40, -8, 0))), -2),
    (dict(pieces=_pieces(ptr=None)), -1), (dict(pieces=_pieces(ptr=FAKE + 1)), -7),
    (dict(x=None), -1), (dict(weight=None), -1), (dict(x=FAKE + 1), -7), (dict(weight=FAKE + 1), -7), (dict(bias=FAKE + 1), -7),
    (dict(shape=dict(B=1, N=2), cu=FAKE + 2), -7),
])
def test_conv_refusals(entry, kw, want):
    assert _conv(entry, **kw) == want


@pytest.mark.parametrize("entry,kw,want", [
    ("fwd", dict(initial=FAKE + 1), -7), ("fwd", dict(final=FAKE + 1), -7),
    ("pool", dict(no_pool=True), -1), ("pool", dict(pool=dict(data=None)), -1), ("pool", dict(pool=dict(indices=None)), -1),
    ("pool", dict(pool=dict(dtype=F32)), -3), ("pool", dict(pool=dict(pool_size=0)), -2),
    ("pool", dict(pool=dict(data=FAKE + 1)), -7), ("pool", dict(pool=dict(indices=FAKE + 2)), -7),
    ("update", dict(no_pool=True), -1), ("update", dict(pool=dict(data=None)), -1),
    ("update", dict(pool=dict(dtype=F32)), -3), ("update", dict(pool=dict(cols=0)), -2),
    ("update", dict(pool=dict(data=FAKE + 1)), -7), ("update", dict(pool=dict(num_accepted=FAKE + 2)), -7),
    ("update", dict(shape=dict(T=0)), 0), ("fwd", dict(shape=dict(B=0, N=0)), 0),
    ("bwd", dict(dx=None), -1), ("bwd", dict(dweight=None), -1), ("bwd", dict(dx=FAKE + 1), -7),
    ("bwd", dict(dweight=FAKE + 2), -7), ("bwd", dict(dbias=FAKE + 2), -7), ("bwd", dict(dinitial=FAKE + 1), -7),
    ("bwd", dict(ws=None), -5), ("bwd", dict(ws=FAKE + 4), -5), ("bwd", dict(ws_bytes=64), -5),
])
def test_conv_refusals_of_one_entry(entry, kw, want):
    assert _conv(entry, **kw) == want


def test_conv_workspace_size():
    size = lambda **kw: gdn.gdn_conv_bwd_workspace_bytes(gdn.gdn_conv_shape(**{**CONV_SHAPE, **kw}))
    assert size(T=0) == 0 and size(W=5) == 0 and size(D=0) == 0 and size(B=-1) == 0
    # W + 1 floats a column for each block of 12 to 256 tokens
    for B, T, D, W in ((1, 1, 32, 4), (2, 5, 33, 2), (4, 4096, 8192, 4), (1, 70000, 64, 3)):
        rows, rest = divmod(size(B=B, T=T, D=D, W=W), 4 * D * (W + 1))
        assert rest == 0 and -(-B * T // 256) <= rows <= -(-B * T // 12)


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------
NORM_SHAPE = dict(rows=8, z_stride=256, D=128, heads=2, dtype=BF, weight_dtype=F32)


def _norm(entry, shape=None, no_shape=False, ws=FAKE, ws_bytes=1 << 30, **ptr):
    s = gdn.gdn_norm_shape(**{**NORM_SHAPE, **(shape or {})})
    names = ("x", "z", "weight", "out", "hidden", "dout", "dhidden", "dx", "dz", "dresidual", "dweight")
    a = {n: ptr.get(n, FAKE) for n in names}
    sp = None if no_shape else ctypes.byref(s)
    if entry == "gated":
        return _lib().gdn_gated_norm(a["x"], a["z"], a["weight"], 1e-6, a["out"], sp, None)
    if entry == "add":
        return _lib().gdn_add_norm(a["x"], a["z"], a["weight"], 1.0, 0.0, 1e-6, a["out"], a["hidden"], sp, None)
    if entry == "gated_bwd":
        return _lib().gdn_gated_norm_bwd(a["x"], a["z"], a["weight"], 1e-6, a["dout"], a["dx"], a["dz"], a["dweight"],
                                         sp, ws, ws_bytes, None)
    return _lib().gdn_add_norm_bwd(a["dout"], a["dhidden"], a["hidden"], a["weight"], 1.0, 0.0, 1e-6, a["dx"],
                                   a["dresidual"], a["dweight"], sp, ws, ws_bytes, None)


@pytest.mark.parametrize("entry", ["gated", "add", "gated_bwd", "add_bwd"])
@pytest.mark.parametrize("kw,want", [
    (dict(no_shape=True), -1), (dict(shape=dict(rows=-1)), -2), (dict(shape=dict(rows=1 << 31)), -2),
    (dict(shape=dict(D=0)), -2), (dict(shape=dict(dtype=3)), -3), (dict(shape=dict(weight_dtype=3)), -3),
    (dict(shape=dict(D=16385, z_stride=1 << 20)), -4), (dict(shape=dict(dtype=F32, weight_dtype=BF)), -4),
    (dict(weight=None), -1), (dict(weight=FAKE + 2), -7),
])
def test_norm_refusals(entry, kw, want):
    assert _norm(entry, **kw) == want


@pytest.mark.parametrize("entry,kw,want", [
    ("gated", dict(shape=dict(D=1025, z_stride=1 << 20)), -4), ("gated_bwd", dict(shape=dict(D=1025, z_stride=1 << 20)), -4),
    ("gated", dict(shape=dict(heads=0)), -2), ("gated", dict(shape=dict(heads=3, z_stride=384)), -2),
    ("gated", dict(shape=dict(z_stride=255)), -2), ("gated", dict(shape=dict(z_stride=(1 << 31) + 1)), -2),
    ("gated", dict(x=None), -1), ("gated", dict(z=None), -1), ("gated", dict(out=None), -1),
    ("gated", dict(x=FAKE + 1), -7), ("gated", dict(z=FAKE + 1), -7), ("gated", dict(out=FAKE + 1), -7),
    ("gated", dict(shape=dict(rows=0), x=None), 0),
    ("add", dict(x=None), -1), ("add", dict(out=None), -1), ("add", dict(hidden=FAKE + 1), -7), ("add", dict(z=FAKE + 1), -7),
    ("add", dict(shape=dict(rows=0), x=None), 0),
    ("gated_bwd", dict(dout=None), -1), ("gated_bwd", dict(dx=None), -1), ("gated_bwd", dict(dz=None), -1),
    ("gated_bwd", dict(dweight=None), -1), ("gated_bwd", dict(dz=FAKE + 1), -7), ("gated_bwd", dict(dweight=FAKE + 2), -7),
    ("gated_bwd", dict(ws=None), -5), ("gated_bwd", dict(ws=FAKE + 8), -5), ("gated_bwd", dict(ws_bytes=16), -5),
    ("add_bwd", dict(dout=None), -1), ("add_bwd", dict(hidden=None), -1), ("add_bwd", dict(dx=None, dresidual=None), -1),
    ("add_bwd", dict(dweight=None), -1), ("add_bwd", dict(dhidden=FAKE + 1), -7), ("add_bwd", dict(dresidual=FAKE + 1), -7),
    ("add_bwd", dict(ws=None), -5), ("add_bwd", dict(ws_bytes=16), -5),
])
def test_norm_refusals_of_one_entry(entry, kw, want):
    assert _norm(entry, **kw) == want


def test_norm_workspace_size():
    size = lambda **kw: gdn.gdn_norm_bwd_workspace_bytes(gdn.gdn_norm_shape(**{**NORM_SHAPE, **kw}))
    assert size(rows=0) == 0 and size(rows=-1) == 0 and size(D=0) == 0 and size(D=16385) == 0
    for rows, D in ((1, 128), (1000, 128), (1 << 20, 64), (1 << 20, 4096)):
        n, rest = divmod(size(rows=rows, D=D), 4 * D)
        assert rest == 0 and 1 <= n <= min(rows, 512)


# ---------------------------------------------------------------------------
# Python wrappers
# ---------------------------------------------------------------------------
def test_wrappers_refuse_cpu_tensors():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    idx = torch.zeros(1, dtype=torch.int32)
    q, v, g = torch.zeros(1, 4, 1, 64), torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2)
    for call in (lambda: gdn.causal_conv1d(x, w), lambda: gdn.causal_conv1d_bwd(x, w, x),
                 lambda: gdn.causal_conv1d_update(x, w, torch.zeros(2, 8, 3), idx),
                 lambda: gdn.fused_gated_rms_norm(x, x, w[:, 0]), lambda: gdn.fused_add_rms_norm(x, x, w[:, 0]),
                 lambda: gdn.fused_gated_rms_norm_bwd(x, x, w[:, 0], x),
                 lambda: gdn.fused_add_rms_norm_bwd(x, x, x, w[:, 0]),
                 lambda: gdn.fused_recurrent_gated_delta_rule_steps(q, q, v, g, g, torch.zeros(2, 2, 64, 64), idx)):
        with pytest.raises(ValueError, match="GPU"):
            call()
