"""Host-side checks of the linear recurrence and of held values (no GPU): every
refused argument of the C entry points.  The argument pointers are never
dereferenced: every call fails a check first, or has nothing to compute."""
import ctypes

import pytest
import torch

import gated_deltanet_chunked_delta_amd as gdn

FAKE = 1 << 20
BF, F32 = gdn.GDN_BF16, gdn.GDN_F32
SHAPE = dict(B=2, T=300, D=64, N=2, dtype=BF, gate_dtype=F32, x_stride=64, g_stride=64, beta_stride=64)


def _lib():
    from gated_deltanet_chunked_delta_amd import _binding_scan
    return _binding_scan._load()


def _ref(s):
    return None if s is None else ctypes.byref(s)


def _scan(entry, shape=None, cu=None, no_shape=False, pool=None, no_pool=False, ws=FAKE, ws_bytes=1 << 30, held=False,
          x8=True, **ptr):
    s = gdn.gdn_scan_shape(**{**SHAPE, **(shape or {})})
    a = {n: ptr.get(n, FAKE) for n in ("x", "g", "beta", "initial", "out", "final", "y", "dout", "dht", "dx", "dg", "dbeta")}
    sp = None if no_shape else ctypes.byref(s)
    if entry == "fwd":
        return _lib().gdn_scan_fwd(a["x"], a["g"], a["beta"], a["initial"], cu, a["out"], a["final"], sp, ws, ws_bytes, None)
    if entry == "pool":
        pl = gdn.gdn_state_pool(**{**dict(data=FAKE, indices=FAKE, pool_size=9, dtype=F32, read_initial=1), **(pool or {})})
        return _lib().gdn_scan_fwd_pool(a["x"], a["g"], a["beta"], None if no_pool else ctypes.byref(pl), cu, a["out"], sp,
                                        ws, ws_bytes, None)
    if entry == "steps":
        pl = gdn.gdn_step_pool(**{**dict(data=FAKE, indices=FAKE, num_accepted=FAKE, pool_size=9, cols=2, dtype=F32), **(pool or {})})
        return _lib().gdn_scan_steps(a["x"], a["g"], a["beta"], None if no_pool else ctypes.byref(pl), cu, a["out"], sp, None)
    h = gdn.gdn_held(ptr.get("codes", FAKE), ptr.get("scales", FAKE))
    return _lib().gdn_scan_bwd(a["x"], a["g"], a["beta"], a["y"], _ref(h if held and x8 else None), _ref(h if held else None),
                               a["dout"], a["dht"], a["initial"], cu, a["dx"], a["dg"], a["dbeta"], a["final"], sp, ws,
                               ws_bytes, None)


EVERY = pytest.mark.parametrize("entry", ["fwd", "pool", "steps", "bwd"])


@EVERY
@pytest.mark.parametrize("kw,want", [
    (dict(no_shape=True), -1), (dict(g=None), -1),
    (dict(shape=dict(N=3)), -2), (dict(cu=FAKE), -2),                        # N != B; B != 1 with cu_seqlens
    (dict(shape=dict(B=1, N=0), cu=FAKE), -2),                               # tokens without a sequence
    (dict(shape=dict(T=-1)), -2), (dict(shape=dict(D=0)), -2), (dict(shape=dict(D=(1 << 26) + 1)), -2),
    (dict(shape=dict(B=1 << 16, T=1 << 15, N=1 << 16)), -2),                 # 2^31 tokens
    (dict(shape=dict(B=1, T=1 << 30, N=1, D=8192, x_stride=8192, g_stride=8192, beta_stride=8192)), -2),   # too many tiles
    (dict(shape=dict(x_stride=63)), -2), (dict(shape=dict(g_stride=0)), -2), (dict(shape=dict(beta_stride=63)), -2),
    (dict(shape=dict(g_stride=(1 << 31) + 1)), -2),
    (dict(shape=dict(dtype=5)), -3), (dict(shape=dict(gate_dtype=-1)), -3),
    (dict(shape=dict(dtype=F32, gate_dtype=BF)), -4),
    (dict(shape=dict(B=1, N=2), cu=FAKE + 2), -7),
    (dict(g=FAKE + 2), -7), (dict(beta=FAKE + 1), -7),
])
def test_scan_refusals(entry, kw, want):
    assert _scan(entry, **kw) == want


@pytest.mark.parametrize("entry,kw,want", [
    ("fwd", dict(x=None), -1), ("fwd", dict(out=None), -1), ("fwd", dict(x=FAKE + 1), -7), ("fwd", dict(final=FAKE + 2), -7),
    ("fwd", dict(ws=None), -5), ("fwd", dict(ws=FAKE + 8), -5), ("fwd", dict(ws_bytes=16), -5),
    ("pool", dict(no_pool=True), -1), ("pool", dict(pool=dict(data=None)), -1), ("pool", dict(pool=dict(indices=None)), -1),
    ("pool", dict(pool=dict(dtype=3)), -3), ("pool", dict(pool=dict(pool_size=0)), -2),
    ("pool", dict(pool=dict(data=FAKE + 2)), -7), ("pool", dict(pool=dict(indices=FAKE + 1)), -7), ("pool", dict(ws=None), -5),
    ("steps", dict(no_pool=True), -1), ("steps", dict(pool=dict(data=None)), -1), ("steps", dict(pool=dict(cols=0)), -2),
    ("steps", dict(pool=dict(pool_size=0)), -2), ("steps", dict(pool=dict(dtype=4)), -3),
    ("steps", dict(pool=dict(data=FAKE + 2)), -7), ("steps", dict(pool=dict(num_accepted=FAKE + 2)), -7),
    ("steps", dict(out=None), -1), ("steps", dict(shape=dict(T=0)), 0),
    ("bwd", dict(y=None), -1), ("bwd", dict(x=None), -1), ("bwd", dict(dout=None), -1), ("bwd", dict(dx=None), -1),
    ("bwd", dict(dg=None), -1), ("bwd", dict(dbeta=None), -1), ("bwd", dict(beta=None), -1),   # dbeta without beta
    ("bwd", dict(held=True, codes=None), -1), ("bwd", dict(held=True, scales=None), -1),
    ("bwd", dict(held=True, x8=False), -1), ("bwd", dict(held=True, scales=FAKE + 1), -7),
    ("bwd", dict(dx=FAKE + 1), -7), ("bwd", dict(dg=FAKE + 2), -7), ("bwd", dict(dht=FAKE + 2), -7),
    ("bwd", dict(ws=None), -5), ("bwd", dict(ws_bytes=64), -5),
    ("fwd", dict(shape=dict(B=0, N=0)), 0), ("bwd", dict(shape=dict(B=0, N=0)), 0),            # nothing to compute
])
def test_scan_refusals_of_one_entry(entry, kw, want):
    assert _scan(entry, **kw) == want


def test_scan_workspace_size():
    need = lambda bwd=False, **kw: gdn.gdn_scan_workspace_bytes(gdn.gdn_scan_shape(**{**SHAPE, **kw}), bwd)  # noqa: E731
    assert need(T=16) == need(T=1, B=1, N=1, bwd=True) == 0           # one tile
    a, b = need(T=4096, D=4096), need(T=8192, D=4096)
    assert 0 < a < b < 2 * a + (1 << 16) and a % 16 == 0
    assert need(T=4096, D=4096, gate_dtype=BF) > 0 and need(T=4096, D=4096, bwd=True) > 0
    for bad in (dict(T=-1), dict(D=0), dict(dtype=9), dict(gate_dtype=9), dict(B=1 << 16, T=1 << 16)):
        assert need(**bad) == 0
    assert _lib().gdn_scan_workspace_bytes(None, 0) == 0


HELD = dict(n=4, D=100, stride=100, value_rows=9, held_rows=7, dtype=BF, bits=8)


def _hold(entry, shape=None, no_shape=False, no_held=False, **ptr):
    s = gdn.gdn_held_shape(**{**HELD, **(shape or {})})
    h = gdn.gdn_held(ptr.get("codes", FAKE), ptr.get("scales", FAKE))
    v, vi, hi = (ptr.get(n, FAKE) for n in ("values", "value_index", "held_index"))
    sp, hp = None if no_shape else ctypes.byref(s), None if no_held else ctypes.byref(h)
    if entry == "hold":
        return _lib().gdn_hold(v, vi, hp, hi, sp, None)
    return _lib().gdn_restore(hp, hi, v, vi, sp, None)


@pytest.mark.parametrize("entry", ["hold", "restore"])
@pytest.mark.parametrize("kw,want", [
    (dict(no_shape=True), -1), (dict(no_held=True), -1), (dict(values=None), -1), (dict(codes=None), -1),
    (dict(scales=None), -1),
    (dict(shape=dict(n=-1)), -2), (dict(shape=dict(D=0)), -2), (dict(shape=dict(D=1 << 31)), -2),
    (dict(shape=dict(stride=99)), -2), (dict(shape=dict(stride=(1 << 31) + 1)), -2), (dict(shape=dict(value_rows=-1)), -2),
    (dict(shape=dict(n=10), value_index=None), -2), (dict(shape=dict(n=8), held_index=None), -2),
    (dict(shape=dict(n=1 << 31)), -2), (dict(shape=dict(n=1 << 20, D=1 << 20, stride=1 << 20)), -2),
    (dict(shape=dict(dtype=2)), -3), (dict(shape=dict(bits=5)), -4), (dict(shape=dict(bits=16)), -4),
    (dict(values=FAKE + 1), -7), (dict(scales=FAKE + 1), -7), (dict(value_index=FAKE + 2), -7), (dict(held_index=FAKE + 1), -7),
    (dict(shape=dict(n=0)), 0),
])
def test_hold_refusals(entry, kw, want):
    assert _hold(entry, **kw) == want


NORM = dict(rows=6, z_stride=256, D=64, heads=2, dtype=BF, weight_dtype=BF)


def _norm(entry, shape=None, ws=FAKE, ws_bytes=1 << 20, no_shape=False, no_x8=False, no_z8=False, **ptr):
    s = gdn.gdn_norm_shape(**{**NORM, **(shape or {})})
    h = gdn.gdn_held(ptr.get("codes", FAKE), ptr.get("scales", FAKE))
    a = {n: ptr.get(n, FAKE) for n in ("x", "z", "weight", "out", "dout", "dx", "dz", "dweight")}
    x8, z8, sp = _ref(None if no_x8 else h), _ref(None if no_z8 else h), None if no_shape else ctypes.byref(s)
    if entry == "fwd":
        return _lib().gdn_gated_norm_hold(a["x"], a["z"], a["weight"], 1e-6, a["out"], x8, z8, sp, None)
    return _lib().gdn_gated_norm_hold_bwd(x8, z8, a["weight"], 1e-6, a["dout"], a["dx"], a["dz"], a["dweight"], sp, ws,
                                          ws_bytes, None)


@pytest.mark.parametrize("entry", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,want", [
    (dict(no_shape=True), -1), (dict(weight=None), -1), (dict(no_x8=True), -1), (dict(no_z8=True), -1),
    (dict(codes=None), -1), (dict(scales=None), -1), (dict(scales=FAKE + 1), -7),
    (dict(shape=dict(rows=-1)), -2), (dict(shape=dict(rows=7)), -2), (dict(shape=dict(heads=0)), -2),
    (dict(shape=dict(z_stride=127)), -2), (dict(shape=dict(dtype=6)), -3), (dict(shape=dict(D=1025, z_stride=4096)), -4),
    (dict(shape=dict(dtype=F32)), -4), (dict(weight=FAKE + 1), -7),
])
def test_norm_refusals(entry, kw, want):
    assert _norm(entry, **kw) == want


@pytest.mark.parametrize("entry,kw,want", [
    ("fwd", dict(x=None), -1), ("fwd", dict(z=None), -1), ("fwd", dict(out=None), -1), ("fwd", dict(x=FAKE + 1), -7),
    ("fwd", dict(shape=dict(rows=0)), 0),
    ("bwd", dict(dout=None), -1), ("bwd", dict(dx=None), -1), ("bwd", dict(dz=None), -1), ("bwd", dict(dweight=None), -1),
    ("bwd", dict(dz=FAKE + 1), -7), ("bwd", dict(dweight=FAKE + 2), -7), ("bwd", dict(ws=None), -5), ("bwd", dict(ws_bytes=8), -5),
])
def test_norm_refusals_of_one_entry(entry, kw, want):
    assert _norm(entry, **kw) == want


def test_wrappers_refuse_cpu_tensors():
    x, i = torch.zeros(2, 4, 32), torch.zeros(2, dtype=torch.int32)
    pool, c = torch.zeros(3, 32), gdn.Checkpoint(torch.zeros(2, 4, 32, dtype=torch.int8), torch.zeros(2, 4, 1, dtype=torch.bfloat16))
    codes, scales = gdn.make_state_cache(pool, 3)
    for call in (lambda: gdn.gated_linear_recurrence(x, x), lambda: gdn.gated_linear_recurrence_steps(x, x, pool, i),
                 lambda: gdn.gated_linear_recurrence_bwd(x, x, x, x), lambda: gdn.checkpoint_activation(x),
                 lambda: gdn.restore_activation(c), lambda: gdn.state_cache_write(pool, i, codes, scales, i),
                 lambda: gdn.state_cache_read(codes, scales, i, pool, i),
                 lambda: gdn.fused_gated_rms_norm_checkpoint(x, x, torch.zeros(32)),
                 lambda: gdn.fused_gated_rms_norm_checkpoint_bwd(c, c, torch.zeros(32), x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
