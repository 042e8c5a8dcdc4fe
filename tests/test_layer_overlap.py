"""Buffers to be written that overlap what a call of the operators around the
delta rule reads, or each other: the Python wrappers refuse them before the
library is called (no GPU; CPU tensors stand for GPU ones)."""
import pytest
import torch

import gated_deltanet_chunked_delta_amd as gdn
from gated_deltanet_chunked_delta_amd import _binding_layer as layer_binding

Z, I32 = torch.zeros, torch.int32


class Called(Exception):
    pass


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def run(*a):
        raise Called
    monkeypatch.setattr(layer_binding, "_gpu", lambda x, n: (-1, layer_binding._DTYPES[x.dtype]))
    monkeypatch.setattr(layer_binding, "_run", run)


def _two(n, shift, *shape):
    """Two contiguous tensors of one shape in a buffer, the second `shift` elements behind the first."""
    buf = Z(n)
    k = Z(shape).numel()
    return buf[:k].view(shape), buf[shift:shift + k].view(shape)


REFUSED = {}


def refused(call):
    REFUSED[call.__name__[1:]] = call


def _conv(x, out=None, **kw):
    return gdn.causal_conv1d(x, Z(8, 4), out=out, **kw)


def _update(x, pool, out, **kw):
    return gdn.causal_conv1d_update(x, Z(8, 4), pool, Z(2, dtype=I32), out=out, **kw)


def _steps(q, k, v, out, pool=None, g=None):
    n = v.shape[2]
    return gdn.fused_recurrent_gated_delta_rule_steps(q, k, v, Z(1, 2, n) if g is None else g, Z(1, 2, n),
                                                      Z(3, n, 64, 64) if pool is None else pool, Z(1, dtype=I32), out=out)


@refused
def _conv_out_is_x():
    x = Z(2, 4, 8)
    _conv(x, out=x)


@refused
def _conv_out_a_row_on():
    x, out = _two(200, 8, 2, 4, 8)
    _conv(x, out=out)


@refused
def _conv_out_in_wider_rows():
    wide = Z(1, 4, 16)
    _conv(wide[..., 8:], out=wide.view(1, 8, 8)[:, 2:6])


@refused
def _conv_parts_overlap():
    a, b = _two(200, 31, 2, 4, 4)
    _conv(Z(2, 4, 8), out=[a, b], split_sizes=(4, 4))


@refused
def _conv_part_twice():
    a = Z(2, 4, 4)
    _conv(Z(2, 4, 8), out=[a, a], split_sizes=(4, 4))


@refused
def _conv_out_over_start():
    buf = Z(200)
    _conv(Z(2, 4, 8), out=buf[:64].view(2, 4, 8), initial_state=buf[63:111].view(2, 8, 3))


@refused
def _conv_out_over_weight():
    buf = Z(200)
    gdn.causal_conv1d(Z(2, 4, 8), buf[:32].view(8, 4), out=buf[16:80].view(2, 4, 8))


@refused
def _conv_final_over_x():
    buf = Z(200)
    _conv(buf[:64].view(2, 4, 8), final_state=buf[60:108].view(2, 8, 3))


@refused
def _conv_final_over_out():
    buf = Z(200)
    _conv(Z(2, 4, 8), out=buf[:64].view(2, 4, 8), final_state=buf[60:108].view(2, 8, 3))


@refused
def _conv_final_partly_start():
    start, final = _two(200, 24, 2, 8, 3)
    _conv(Z(2, 4, 8), initial_state=start, final_state=final)


@refused
def _conv_out_over_pool():
    buf = Z(200)
    _conv(Z(2, 4, 8), out=buf[70:134].view(2, 4, 8), conv_state_pool=buf[:72].view(3, 8, 3), conv_state_indices=Z(2, dtype=I32))


@refused
def _update_out_is_x():
    x = Z(2, 4, 8)
    _update(x, Z(3, 8, 3), x)


@refused
def _update_single_out_is_x():
    x = Z(2, 8)
    _update(x, Z(3, 8, 3), x)


@refused
def _update_out_over_pool():
    buf = Z(200)
    _update(Z(2, 4, 8), buf[:72].view(3, 8, 3), buf[70:134].view(2, 4, 8))


def _steps_out_is(name):
    def call():
        t = {n: Z(1, 2, 2, 64) for n in "qkv"}
        _steps(t["q"], t["k"], t["v"], t[name])
    return call


@refused
def _steps_out_partly_v():
    v, out = _two(600, 64, 1, 2, 2, 64)
    _steps(Z(1, 2, 1, 64), Z(1, 2, 1, 64), v, out)


@refused
def _steps_out_over_pool():
    pool = Z(3, 2, 64, 64)
    _steps(Z(1, 2, 1, 64), Z(1, 2, 1, 64), Z(1, 2, 2, 64), pool.view(-1)[:256].view(1, 2, 2, 64), pool)


@refused
def _steps_out_over_gates():
    buf = Z(300)
    _steps(Z(1, 2, 1, 64), Z(1, 2, 1, 64), Z(1, 2, 2, 64), buf[:256].view(1, 2, 2, 64), g=buf[252:256].view(1, 2, 2))


def _gated_out_a_row_on(which):
    def call():
        t, out = _two(200, 8, 4, 8)
        gdn.fused_gated_rms_norm(*((t, Z(4, 8)) if which == "x" else (Z(4, 8), t)), Z(8), out=out)
    return call


@refused
def _gated_out_in_wide_z():
    wide = Z(4, 16)
    gdn.fused_gated_rms_norm(Z(4, 8), wide[:, 8:], Z(8), out=wide.view(8, 8)[:4])


@refused
def _gated_out_over_weight():
    buf = Z(64)
    gdn.fused_gated_rms_norm(Z(4, 8), Z(4, 8), buf[:8], out=buf[4:36].view(4, 8))


@refused
def _add_out_a_row_on():
    x, out = _two(200, 8, 4, 8)
    gdn.fused_add_rms_norm(x, None, Z(8), out=out)


@refused
def _add_hidden_partly_residual():
    res, hidden = _two(200, 8, 4, 8)
    gdn.fused_add_rms_norm(Z(4, 8), res, Z(8), hidden=hidden)


@refused
def _add_out_is_hidden():
    t = Z(4, 8)
    gdn.fused_add_rms_norm(Z(4, 8), Z(4, 8), Z(8), out=t, hidden=t)


REFUSED.update(steps_out_is_q=_steps_out_is("q"), steps_out_is_k=_steps_out_is("k"),
               gated_out_a_row_on_x=_gated_out_a_row_on("x"), gated_out_a_row_on_z=_gated_out_a_row_on("z"))


@pytest.mark.parametrize("name", list(REFUSED))
def test_overlaps_are_refused(name):
    with pytest.raises(ValueError, match="overlap"):
        REFUSED[name]()


def _parts_of_one_buffer():
    buf = Z(3, 2, 4, 8)
    _conv(buf[0], out=buf[1])


def _pieces_side_by_side():
    a, b = _two(200, 32, 2, 4, 4)
    _conv(Z(2, 4, 8), out=[a, b], split_sizes=(4, 4))


def _final_is_start():
    h = Z(2, 8, 3)
    _conv(Z(2, 4, 8), initial_state=h, final_state=h, out=Z(2, 4, 8))


def _one_token_beside_its_row():
    wide = Z(1, 1, 16)
    _conv(wide[..., 8:], out=wide[..., :8])


def _empty():
    _conv(Z(2, 0, 8), out=Z(2, 0, 8), initial_state=Z(2, 8, 3))


def _hidden_is_residual():
    res = Z(4, 8)
    gdn.fused_add_rms_norm(Z(4, 8), res, Z(8), hidden=res, out=Z(4, 8))


def _update_own_out():
    _update(Z(2, 4, 8), Z(3, 8, 3), Z(2, 4, 8))


def _steps_own_out():
    _steps(Z(1, 2, 1, 64), Z(1, 2, 1, 64), Z(1, 2, 2, 64), Z(1, 2, 2, 64))


ALLOWED = [_parts_of_one_buffer, _pieces_side_by_side, _final_is_start, _one_token_beside_its_row, _empty, _hidden_is_residual,
           _update_own_out, _steps_own_out]


@pytest.mark.parametrize("call", ALLOWED, ids=lambda f: f.__name__[1:])
def test_buffers_apart_reach_the_library(call):
    with pytest.raises(Called):
        call()
