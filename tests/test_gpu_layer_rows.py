"""Rows of the RMS norms that hold an infinity, or whose squares overflow fp32:
the definition's values, whatever the row's length (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
INF = float("inf")
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _rows(D, dtype):
    """Ones with one infinity a row, at the row's ends and on both sides of where its last whole vectors meet; a
    row without one; a row whose squares overflow."""
    at = sorted({0, D // 2, D - 1, max(D - 2, 0), max(D - 7, 0), max(D - 8, 0), D // 8 * 8 - 1 if D >= 8 else 0,
                 min(D // 8 * 8, D - 1)})
    x = torch.ones(len(at) + 2, D, dtype=dtype, device=DEV)
    for i, a in enumerate(at):
        x[i, a] = -INF if i % 2 else INF
    x[-1, D // 3:] = 3e38 if dtype == torch.float32 else 1e38
    return x, at


def _check(y, at, finite):
    """An infinite sum of squares makes r = 0: zeros, and inf * 0 = NaN at the infinity."""
    for i, a in enumerate(at):
        assert bool(torch.isnan(y[i, a])), (i, a)
        rest = torch.cat([y[i, :a], y[i, a + 1:]])
        assert not bool(torch.isnan(rest).any()) and not bool(rest.any()), f"infinity at {a}: the row's other elements"
    assert torch.equal(y[len(at)], finite)
    assert not bool(y[-1].any()), "overflowing squares"


@TYPES
@pytest.mark.parametrize("D", [8, 13, 15, 64, 125, 187, 256, 509, 1000, 1021, 1024])
def test_gated_norm_rows_with_an_infinity(D, dtype):
    gdn = _gdn()
    x, at = _rows(D, dtype)
    z, w = torch.ones_like(x), torch.ones(D, dtype=dtype, device=DEV)
    n = len(at)
    _check(gdn.fused_gated_rms_norm(x, z, w), at, gdn.fused_gated_rms_norm(x[n:n + 1], z[n:n + 1], w)[0])


@TYPES
@pytest.mark.parametrize("D", [13, 187, 1021, 1027, 2048, 2049, 4093, 5001, 8192, 9001, 16383])
def test_add_norm_rows_with_an_infinity(D, dtype):
    gdn = _gdn()
    x, at = _rows(D, dtype)
    w = torch.ones(D, dtype=dtype, device=DEV)
    y, hidden = gdn.fused_add_rms_norm(x, torch.zeros_like(x), w)
    n = len(at)
    _check(y, at, gdn.fused_add_rms_norm(x[n:n + 1], None, w)[0][0])
    assert torch.equal(hidden, x)
