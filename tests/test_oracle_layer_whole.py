"""The whole-tensor forms in oracle/layer_whole.py equal the definitions in
oracle/layer.py, values and magnitudes (no GPU).  Both are sums of at most a few
hundred float64 terms of order one: 1e-11 is far above their rounding."""
import numpy as np
import pytest
import torch

from oracle import layer, layer_whole

LENS = [3, 0, 1, 2, 17, 0, 4, 1]


def _close(got, want):
    np.testing.assert_allclose(got.numpy().reshape(want.shape), want, rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("start", [True, False])
def test_conv(W, silu, start):
    gen = torch.Generator().manual_seed(W)
    D, T = 5, sum(LENS)
    r = lambda *shape: torch.randn(*shape, generator=gen, dtype=torch.float64)
    x, w, b, dy = r(1, T, D), r(D, W), r(D) if start else None, r(1, T, D)
    h0 = r(len(LENS), D, W - 1) if start else None
    cu = [sum(LENS[:i]) for i in range(len(LENS) + 1)]
    for got, want in zip(layer_whole.conv(x, w, b, h0, LENS, silu), layer.conv(x, w, b, h0, cu, silu)):
        _close(got, want)
    got, want = layer_whole.conv_bwd(x, w, dy, b, h0, LENS, silu), layer.conv_bwd(x, w, dy, b, h0, cu, silu)
    for name in want:
        for g, v in zip(got[name], want[name]):
            _close(g, v)


def test_norms():
    gen = torch.Generator().manual_seed(5)
    x, z, dy, dh = (torch.randn(4, 3, 9, generator=gen, dtype=torch.float64) for _ in range(4))
    w = torch.randn(9, generator=gen, dtype=torch.float64)
    for got, want in zip(layer_whole.gated_norm(x, z, w), layer.gated_norm(x, z, w)):
        _close(got, want)
    kw = dict(residual_scale=-0.7, weight_offset=1.0)
    for res, more in ((z, kw), (None, {})):
        got, want = layer_whole.add_norm(x, res, w, **more), layer.add_norm(x, res, w, **more)
        for g, v in zip(got, want):
            _close(g, v)
    pairs = [(layer_whole.gated_norm_bwd(x, z, w, dy), layer.gated_norm_bwd(x, z, w, dy)),
             (layer_whole.add_norm_bwd(dy, dh, x, w, **kw), layer.add_norm_bwd(dy, dh, x, w, **kw)),
             (layer_whole.add_norm_bwd(dy, None, x, w), layer.add_norm_bwd(dy, None, x, w))]
    for got, want in pairs:
        for name in want:
            for g, v in zip(got[name], want[name]):
                _close(g, v)
