"""Arguments that the Python wrappers of the linear recurrence and of held values
refuse (no GPU): each raises ValueError before the library is called."""
import pytest
import torch

import gated_deltanet_chunked_delta_amd as gdn
from gated_deltanet_chunked_delta_amd import _binding_layer, _binding_scan

BIG = 1 << 31
Z, BF, F32, I32, I8, U8 = torch.zeros, torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.uint8


def _rec(x=(2, 4, 8), g=None, dt=F32, gdt=None, **kw):
    return gdn.gated_linear_recurrence(Z(x, dtype=dt), Z(g or x, dtype=gdt or dt), **kw)


def _steps(x=(2, 4, 8), g=None, pool=(5, 8), idx=None, pdt=F32, **kw):
    return gdn.gated_linear_recurrence_steps(Z(x), Z(g or x), Z(pool, dtype=pdt), Z(2, dtype=I32) if idx is None else idx, **kw)


def _bwd(x=(2, 4, 8), g=None, y=None, dy=(2, 4, 8), beta=(2, 4, 8), dt=F32, **kw):
    val = lambda t: t if t is None or isinstance(t, (torch.Tensor, gdn.Checkpoint)) else Z(t, dtype=dt)  # noqa: E731
    return gdn.gated_linear_recurrence_bwd(val(x), Z(g or dy, dtype=dt), val(dy if y is None else y), Z(dy, dtype=dt),
                                           val(beta), **kw)


def _ck(shape=(2, 4, 8), groups=1, cdt=I8, sdt=BF):
    return gdn.Checkpoint(Z(shape, dtype=cdt), Z((*shape[:-1], groups), dtype=sdt))


def _cache(pool=(3, 2, 40), codes=(4, 80), scales=(4, 3), pi=None, ci=None, cdt=I8, sdt=BF, pdt=F32, read=False):
    a = (Z(pool, dtype=pdt) if isinstance(pool, tuple) else pool, Z(2, dtype=I32) if pi is None else pi,
         Z(codes, dtype=cdt), Z(scales, dtype=sdt), Z(2, dtype=I32) if ci is None else ci)
    return gdn.state_cache_read(a[2], a[3], a[4], a[0], a[1]) if read else gdn.state_cache_write(*a)


def _one(n=64, dtype=U8):
    return Z(n, dtype=dtype)


CU = torch.tensor([0, 4], dtype=I32)
SHARED = Z(4, 40)

REFUSED = {
    "x of two dimensions": lambda: _rec(x=(4, 8)),
    "x without channels": lambda: _rec(x=(2, 4, 0)),
    "x beyond 32 bits": lambda: gdn.gated_linear_recurrence(Z(1).expand(1, BIG, 1), Z(1).expand(1, BIG, 1)),
    "half precision": lambda: _rec(dt=torch.float16),
    "g of another shape": lambda: _rec(g=(2, 4, 9)),
    "g of a narrower type": lambda: _rec(gdt=BF),
    "beta of another shape": lambda: _rec(beta=Z(2, 3, 8)),
    "beta of another type than g": lambda: _rec(dt=BF, gdt=F32, beta=Z(2, 4, 8, dtype=BF)),
    "initial state of another shape": lambda: _rec(initial_state=Z(3, 8)),
    "initial state in bf16": lambda: _rec(initial_state=Z(2, 8, dtype=BF)),
    "final state of another type": lambda: _rec(final_state=Z(2, 8, dtype=BF)),
    "final state not contiguous": lambda: _rec(final_state=Z(8, 2).t()),
    "cu_seqlens with rows": lambda: _rec(cu_seqlens=CU),
    "cu_seqlens of 64 bits": lambda: _rec(x=(1, 4, 8), cu_seqlens=CU.long()),
    "cu_seqlens without entries": lambda: _rec(x=(1, 4, 8), cu_seqlens=CU[:0]),
    "out of another shape": lambda: _rec(out=Z(2, 4, 9)),
    "out of another type": lambda: _rec(out=Z(2, 4, 8, dtype=BF)),
    "pool with an initial state": lambda: _rec(state_pool=Z(5, 8), state_indices=Z(2, dtype=I32), initial_state=Z(2, 8)),
    "pool of other channels": lambda: _rec(state_pool=Z(5, 9), state_indices=Z(2, dtype=I32)),
    "pool of a third type": lambda: _rec(state_pool=Z(5, 8, dtype=torch.float16), state_indices=Z(2, dtype=I32)),
    "pool without slots named": lambda: _rec(state_pool=Z(5, 8)),
    "pool slots of other sequences": lambda: _rec(state_pool=Z(5, 8), state_indices=Z(3, dtype=I32)),
    "pool slots in columns": lambda: _rec(state_pool=Z(5, 8), state_indices=Z(2, 1, dtype=I32)),
    "workspace too small": lambda: _rec(x=(1, 4096, 8), workspace=_one()),
    "workspace not contiguous": lambda: _rec(x=(1, 4096, 8), workspace=_one(1 << 22).view(2, -1).t()),
    "steps g of another shape": lambda: _steps(g=(2, 4, 9)),
    "steps flat x, g with tokens": lambda: _steps(x=(2, 8), g=(2, 1, 8)),
    "steps flat x with cu_seqlens": lambda: _steps(x=(2, 8), cu_seqlens=CU),
    "steps pool of other channels": lambda: _steps(pool=(5, 9)),
    "steps pool of a third type": lambda: _steps(pdt=torch.float16),
    "steps slots of 64 bits": lambda: _steps(idx=Z(2, dtype=torch.int64)),
    "steps slots without columns": lambda: _steps(idx=Z(2, 0, dtype=I32)),
    "steps counts of other sequences": lambda: _steps(num_accepted=Z(3, dtype=I32)),
    "steps out of another shape": lambda: _steps(out=Z(2, 4, 9)),
    "gradient of two dimensions": lambda: _bwd(dy=(4, 8), beta=None, x=None),
    "gradient y of another shape": lambda: _bwd(y=(2, 4, 9)),
    "gradient x of another shape": lambda: _bwd(x=(2, 4, 9)),
    "gradient with beta without x": lambda: _bwd(x=None),
    "gradient of a checkpoint and a tensor": lambda: _bwd(y=_ck()),
    "gradient of a tensor and a checkpoint": lambda: _bwd(x=_ck()),
    "gradient of codes of other values": lambda: _bwd(x=_ck((2, 4, 9)), y=_ck()),
    "gradient of scales of other groups": lambda: _bwd(x=_ck(), y=_ck(groups=2)),
    # as many scales as rows of 62 have, but of groups that end with each 31 values
    "gradient of codes of two heads of 31": lambda: _bwd(x=(1, 4, 62), dy=(1, 4, 62), beta=None, y=_ck((1, 4, 2, 31))),
    "gradient of codes of longer rows": lambda: _bwd(x=(1, 2, 31), dy=(1, 2, 31), beta=None, y=_ck((1, 62), 2)),
    "norm gradient of codes of two heads of 31": lambda: gdn.fused_gated_rms_norm_checkpoint_bwd(
        _ck((3, 2, 31)), _ck((3, 62), 2), Z(62), Z(3, 62)),
    "gradient of uint8 codes": lambda: _bwd(x=_ck(cdt=U8), y=_ck()),
    "gradient of fp32 scales": lambda: _bwd(x=_ck(), y=_ck(sdt=F32)),
    "gradient dht of another shape": lambda: _bwd(dht=Z(2, 9)),
    "gradient dht in bf16": lambda: _bwd(dht=Z(2, 8, dtype=BF)),
    "gradient initial state of another shape": lambda: _bwd(initial_state=Z(1, 8)),
    "gradient beta of another shape": lambda: _bwd(beta=(2, 4, 1)),
    "gradient workspace too small": lambda: _bwd(x=(1, 4096, 8), dy=(1, 4096, 8), beta=(1, 4096, 8), workspace=_one()),
    "checkpoint of a number": lambda: gdn.checkpoint_activation(Z(())),
    "checkpoint of empty rows": lambda: gdn.checkpoint_activation(Z(3, 0)),
    "checkpoint in half precision": lambda: gdn.checkpoint_activation(Z(3, 8, dtype=torch.float16)),
    "restored to half precision": lambda: gdn.restore_activation(_ck(), torch.float16),
    "restored from other scales": lambda: gdn.restore_activation(_ck(groups=3)),
    "restored into another shape": lambda: gdn.restore_activation(_ck(), out=Z(2, 4, 9, dtype=BF)),
    "cache of 5 bits": lambda: gdn.make_state_cache(Z(3, 4), 2, 5),
    "cache for a pool without slots": lambda: gdn.make_state_cache(Z(0, 4), 2),
    "cache codes of another length": lambda: _cache(codes=(4, 79)),
    "cache codes of 4 bits of another length": lambda: _cache(codes=(4, 41), cdt=U8),
    "cache codes of a third type": lambda: _cache(cdt=torch.int16),
    "cache scales of another length": lambda: _cache(scales=(4, 2)),
    "cache scales of other slots": lambda: _cache(scales=(5, 3)),
    "cache scales in fp32": lambda: _cache(sdt=F32),
    "cache pool not contiguous": lambda: _cache(pool=Z(2, 40, 3).transpose(0, 2)),
    "cache pool without slots": lambda: _cache(pool=(0, 2, 40)),
    "cache slots of different numbers": lambda: _cache(ci=Z(3, dtype=I32)),
    "cache slots of 64 bits": lambda: _cache(pi=Z(2, dtype=torch.int64), ci=Z(2, dtype=torch.int64)),
    "cache read into half precision": lambda: _cache(pdt=torch.float16, read=True),
    "norm z of another shape": lambda: gdn.fused_gated_rms_norm_checkpoint(Z(2, 8), Z(2, 7), Z(8)),
    "norm weight of another length": lambda: gdn.fused_gated_rms_norm_checkpoint(Z(2, 8), Z(2, 8), Z(7)),
    "norm out of another type": lambda: gdn.fused_gated_rms_norm_checkpoint(Z(2, 8), Z(2, 8), Z(8), out=Z(2, 8, dtype=BF)),
    "norm gradient of other rows": lambda: gdn.fused_gated_rms_norm_checkpoint_bwd(_ck((3, 8)), _ck((2, 8)), Z(8), Z(2, 8)),
    "norm gradient of other groups": lambda: gdn.fused_gated_rms_norm_checkpoint_bwd(_ck((2, 8)), _ck((2, 8), 2), Z(8), Z(2, 8)),
    "norm gradient workspace too small": lambda: gdn.fused_gated_rms_norm_checkpoint_bwd(_ck((2, 8)), _ck((2, 8)), Z(8), Z(2, 8),
                                                                                         workspace=_one(1)),
}


def _overlaps():
    b = Z(4096)
    x, g, s = b[:64].view(2, 4, 8), Z(2, 4, 8), b[100:116].view(2, 8)
    i, one = Z(2, dtype=I32), Z(2, 80)
    raw = Z(400, dtype=torch.int16)
    codes8, scales = raw.view(I8)[:160].view(2, 80), raw.view(BF)[70:76].view(2, 3)
    pool = raw.view(F32)[:160].view(2, 80)
    return {
        "out over x": lambda: gdn.gated_linear_recurrence(x, g, out=x),
        "out over the initial state": lambda: gdn.gated_linear_recurrence(g, g, initial_state=s, out=b[64:128].view(2, 4, 8)),
        "final state over x": lambda: gdn.gated_linear_recurrence(x, g, final_state=b[60:76].view(2, 8)),
        "final state over a part of the initial one": lambda: gdn.gated_linear_recurrence(g, g, initial_state=s,
                                                                                          final_state=b[104:120].view(2, 8)),
        "out over the pool": lambda: gdn.gated_linear_recurrence_steps(g, g, b[:40].view(5, 8), i, out=x),
        "scales inside codes": lambda: gdn.state_cache_write(one, i, codes8, scales, i),
        "pool inside codes": lambda: gdn.state_cache_read(codes8, Z(2, 3, dtype=BF), i, pool, i),
        "norm out over x": lambda: gdn.fused_gated_rms_norm_checkpoint(x, g, Z(8), out=x),
    }


REFUSED.update(_overlaps())


@pytest.mark.parametrize("name", list(REFUSED))
def test_wrappers_refuse(name, monkeypatch):
    """CPU tensors stand for GPU ones: device number -1 on all of them."""
    real = _binding_layer._gpu
    fake = lambda x, n: (-1, _binding_layer._DTYPES[x.dtype]) if x.dtype in _binding_layer._DTYPES else real(x, n)  # noqa: E731
    for m in (_binding_layer, _binding_scan):
        monkeypatch.setattr(m, "_gpu", fake)
        monkeypatch.setattr(m, "_run", lambda *a: pytest.fail("the library was called"))
    monkeypatch.setattr(_binding_scan, "_device", lambda t: -1)
    with pytest.raises(ValueError):
        REFUSED[name]()
