"""A caller's workspace is used or refused, never replaced by a new one without
a word (no GPU; CPU tensors stand for GPU ones: device number -1)."""
import pytest
import torch

import gated_deltanet_chunked_delta_amd as gdn
from gated_deltanet_chunked_delta_amd import _binding_layer as layer_binding

Z = torch.zeros
X, W, D = Z(2, 40, 8), Z(8, 4), Z(8)

CALLS = {
    "conv": (lambda ws: gdn.causal_conv1d_bwd(X, W, X, workspace=ws),
             lambda: gdn.gdn_conv_bwd_workspace_bytes(gdn.gdn_conv_shape(2, 40, 8, 4, 2, 1, 1, 8))),
    "gated": (lambda ws: gdn.fused_gated_rms_norm_bwd(X, X, D, X, workspace=ws),
              lambda: gdn.gdn_norm_bwd_workspace_bytes(gdn.gdn_norm_shape(80, 8, 8, 1, 1, 1))),
    "add": (lambda ws: gdn.fused_add_rms_norm_bwd(X, None, X, D, workspace=ws),
            lambda: gdn.gdn_norm_bwd_workspace_bytes(gdn.gdn_norm_shape(80, 8, 8, 1, 1, 1))),
}


@pytest.fixture
def given(monkeypatch):
    """The (pointer, bytes) that reach the library."""
    seen = []
    monkeypatch.setattr(layer_binding, "_gpu", lambda x, n: (-1, layer_binding._DTYPES[x.dtype]))
    monkeypatch.setattr(layer_binding, "_run", lambda dev, fn, *a: seen.append(a[-2:]))
    return seen


@pytest.mark.parametrize("name", list(CALLS))
def test_workspace_is_used(name, given):
    call, need = CALLS[name]
    for extra in (0, 100):
        ws = Z(need() + extra, dtype=torch.uint8)
        call(ws)
        assert given[-1][0] == ws.data_ptr() and given[-1][1] == need()
    call(None)
    assert given[-1][1] == need() and given[-1][0] != 0


@pytest.mark.parametrize("name", list(CALLS))
def test_workspace_is_refused(name, given):
    call, need = CALLS[name]
    for ws, why in ((Z(need() - 1, dtype=torch.uint8), "bytes"), (Z(2 * need(), dtype=torch.uint8)[::2], "contiguous"),
                    (Z(need() - 2, dtype=torch.uint8)[::2], "contiguous")):
        with pytest.raises(ValueError, match=why):
            call(ws)
    assert not given


@pytest.mark.parametrize("size", [64, 1])
def test_workspace_of_another_device_is_refused(size):
    with pytest.raises(ValueError, match="cuda:0"):
        layer_binding._workspace(Z(size, dtype=torch.uint8), 64, 0, X)
