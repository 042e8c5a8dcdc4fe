"""Arguments that the Python wrappers of the operators around the delta rule
refuse (no GPU): each raises ValueError before the library is called."""
import pytest
import torch

import gated_deltanet_chunked_delta_amd as gdn
from gated_deltanet_chunked_delta_amd import _binding_layer as layer_binding

BIG = 1 << 31
Z, BF, I32 = torch.zeros, torch.bfloat16, torch.int32


def _steps(q=(2, 4, 1, 64), k=None, v=(2, 4, 2, 64), g=(2, 4, 2), beta=None, pool=(3, 2, 64, 64), idx=None, dt=torch.float32,
           kdt=None, pdt=torch.float32, **kw):
    return gdn.fused_recurrent_gated_delta_rule_steps(
        Z(q, dtype=dt), Z(k or q, dtype=kdt or dt), Z(v, dtype=dt), None if g is None else Z(g),
        None if g is None else Z(beta or g), Z(pool, dtype=pdt), Z(2, dtype=I32) if idx is None else idx, **kw)


def _gates(n=16, dt=torch.float32, hv=2):
    return {"A_log": Z(hv), "dt_bias": Z(hv), "a_raw": Z(n, dtype=dt), "b_raw": Z(n, dtype=dt)}


def _conv(x=(2, 4, 8), w=(8, 4), **kw):
    return gdn.causal_conv1d(x if isinstance(x, torch.Tensor) else Z(x), w if isinstance(w, torch.Tensor) else Z(w), **kw)


def _update(x=(2, 4, 8), pool=(3, 8, 3), idx=None, **kw):
    return gdn.causal_conv1d_update(Z(x), Z(8, 4), pool if isinstance(pool, torch.Tensor) else Z(pool),
                                    Z(2, dtype=I32) if idx is None else idx, **kw)


def _wide(*shape):   # sizes beyond 32 bits without their memory
    return Z(1).expand(shape)


REFUSED = {
    "steps q of three dimensions": lambda: _steps(q=(2, 4, 64)),
    "steps k of another shape": lambda: _steps(k=(2, 4, 2, 64)),
    "steps v of other tokens": lambda: _steps(v=(2, 5, 2, 64)),
    "steps k of another type": lambda: _steps(kdt=BF),
    "steps half precision": lambda: _steps(dt=torch.float16),
    "steps g of another shape": lambda: _steps(g=(2, 4, 1)),
    "steps beta of another shape": lambda: _steps(beta=(2, 4, 1)),
    "steps without gates": lambda: _steps(g=None),
    "steps with both kinds of gates": lambda: _steps(**_gates()),
    "steps gates of other heads": lambda: _steps(g=None, **_gates(hv=3)),
    "steps gates of other sizes": lambda: _steps(g=None, **_gates(15)),
    "steps gates of another type": lambda: _steps(g=None, **_gates(dt=BF)),
    "steps pool of other heads": lambda: _steps(pool=(3, 1, 64, 64)),
    "steps pool of a third type": lambda: _steps(pdt=torch.float16),
    "steps slots of 64 bits": lambda: _steps(idx=Z(2, dtype=torch.int64)),
    "steps slots of other sequences": lambda: _steps(idx=Z(3, dtype=I32)),
    "steps slots without columns": lambda: _steps(idx=Z(2, 0, dtype=I32)),
    "steps counts of other sequences": lambda: _steps(num_accepted=Z(3, dtype=I32)),
    "steps counts of 64 bits": lambda: _steps(num_accepted=Z(2, dtype=torch.int64)),
    "steps cu_seqlens with rows": lambda: _steps(cu_seqlens=Z(3, dtype=I32)),
    "steps out of another shape": lambda: _steps(out=Z(2, 4, 2, 65)),
    "steps out not contiguous": lambda: _steps(out=Z(2, 4, 64, 2).transpose(2, 3)),
    "conv x of two dimensions": lambda: _conv(x=(4, 8)),
    "conv weight of other columns": lambda: _conv(w=(9, 4)),
    "conv weight of a third type": lambda: _conv(w=Z(8, 4, dtype=BF)),
    "conv bias of another type": lambda: _conv(x=Z(2, 4, 8, dtype=BF), w=Z(8, 4, dtype=BF), bias=Z(8)),
    "conv bias of another shape": lambda: _conv(bias=Z(7)),
    "conv another activation": lambda: _conv(activation="relu"),
    "conv start of another shape": lambda: _conv(initial_state=Z(2, 8, 4)),
    "conv start of another type": lambda: _conv(initial_state=Z(2, 8, 3, dtype=BF)),
    "conv final of another shape": lambda: _conv(final_state=Z(1, 8, 3)),
    "conv sizes of another sum": lambda: _conv(split_sizes=(4, 3)),
    "conv negative size": lambda: _conv(split_sizes=(9, -1)),
    "conv four parts": lambda: _conv(split_sizes=(2, 2, 2, 2)),
    "conv out of fewer parts": lambda: _conv(split_sizes=(4, 4), out=[Z(2, 4, 4)]),
    "conv out of another shape": lambda: _conv(out=Z(2, 4, 7)),
    "conv cu_seqlens of 64 bits": lambda: _conv(x=(1, 4, 8), cu_seqlens=Z(3, dtype=torch.int64)),
    "conv cu_seqlens empty": lambda: _conv(x=(1, 4, 8), cu_seqlens=Z(0, dtype=I32)),
    "conv pool and start": lambda: _conv(conv_state_pool=Z(3, 8, 3), conv_state_indices=Z(2, dtype=I32), initial_state=Z(2, 8, 3)),
    "conv pool without slots": lambda: _conv(conv_state_pool=Z(3, 8, 3)),
    "conv pool with columns of slots": lambda: _conv(conv_state_pool=Z(3, 8, 3), conv_state_indices=Z(2, 1, dtype=I32)),
    "conv tokens beyond 32 bits": lambda: _conv(x=_wide(1, 2 * BIG + 4, 8)),
    "conv rows beyond 32 bits": lambda: _conv(x=_wide(2 * BIG + 2, 1, 8)),
    "conv columns beyond 32 bits": lambda: _conv(x=_wide(1, 4, 2 * BIG + 8), w=_wide(2 * BIG + 8, 4)),
    "update cu_seqlens with single tokens": lambda: _update(x=(2, 8), cu_seqlens=Z(3, dtype=I32)),
    "update pool of another type": lambda: _update(pool=Z(3, 8, 3, dtype=BF)),
    "update pool of another width": lambda: _update(pool=(3, 8, 2)),
    "update pool not contiguous": lambda: _update(pool=Z(3, 3, 8).transpose(1, 2)),
    "update slots of other sequences": lambda: _update(idx=Z(3, dtype=I32)),
    "update slots beyond 32 bits": lambda: _update(idx=Z(1, dtype=I32).expand(2, BIG)),
    "conv gradient of another shape": lambda: gdn.causal_conv1d_bwd(Z(2, 4, 8), Z(8, 4), Z(2, 4, 7)),
    "conv gradient of another type": lambda: gdn.causal_conv1d_bwd(Z(2, 4, 8), Z(8, 4), Z(2, 4, 8, dtype=BF)),
    "gated norm z of another shape": lambda: gdn.fused_gated_rms_norm(Z(2, 8), Z(3, 8), Z(8)),
    "gated norm z of another type": lambda: gdn.fused_gated_rms_norm(Z(2, 8), Z(2, 8, dtype=BF), Z(8)),
    "gated norm weight of another size": lambda: gdn.fused_gated_rms_norm(Z(2, 8), Z(2, 8), Z(7)),
    "gated norm weight of a third type": lambda: gdn.fused_gated_rms_norm(Z(2, 8), Z(2, 8), Z(8, dtype=BF)),
    "gated norm scalar": lambda: gdn.fused_gated_rms_norm(Z(()), Z(()), Z(1)),
    "gated norm out of another type": lambda: gdn.fused_gated_rms_norm(Z(2, 8), Z(2, 8), Z(8), out=Z(2, 8, dtype=BF)),
    "gated norm gradient of another shape": lambda: gdn.fused_gated_rms_norm_bwd(Z(2, 8), Z(2, 8), Z(8), Z(2, 7)),
    "norm residual of another shape": lambda: gdn.fused_add_rms_norm(Z(2, 8), Z(1, 8), Z(8)),
    "norm hidden not contiguous": lambda: gdn.fused_add_rms_norm(Z(2, 8), None, Z(8), hidden=Z(8, 2).t()),
    "norm of no elements": lambda: gdn.fused_add_rms_norm(Z(2, 0), None, Z(0)),
    "norm elements beyond 32 bits": lambda: gdn.fused_add_rms_norm(_wide(1, 2 * BIG + 8), None, _wide(2 * BIG + 8)),
    "norm gradient of another type": lambda: gdn.fused_add_rms_norm_bwd(Z(2, 8, dtype=BF), None, Z(2, 8), Z(8)),
    "norm dhidden of another shape": lambda: gdn.fused_add_rms_norm_bwd(Z(2, 8), Z(2, 7), Z(2, 8), Z(8)),
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_wrappers_refuse(name, monkeypatch):
    """Arguments that do not fit raise ValueError before any call of the library
    (CPU tensors stand for GPU ones: device number -1 on all of them)."""
    real = layer_binding._gpu
    monkeypatch.setattr(layer_binding, "_gpu", lambda x, n: (-1, layer_binding._DTYPES[x.dtype]) if x.dtype in
                        layer_binding._DTYPES else real(x, n))
    monkeypatch.setattr(layer_binding, "_run", lambda *a: pytest.fail("the library was called"))
    with pytest.raises(ValueError):
        REFUSED[name]()
