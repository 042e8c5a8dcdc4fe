"""The gated linear recurrence of few channels without beta: a channel a lane and four strips
of tokens a wave, forward, from tensors and from checkpoints backward, and token by token."""
import numpy as np
import pytest
import torch

from oracle import scan as orc

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
KINDS = pytest.mark.parametrize("dtype,gate", [(BF, F32), (BF, BF), (F32, F32)], ids=["bf16_fp32", "bf16", "fp32"])


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _near(name, got, ref, mag, c):
    """The bar of the recurrence's other tests: c roundings of an fp32 evaluation, and that to the output's type."""
    half = torch.finfo(got.dtype).eps / 2
    tol = c * 2.0 ** -24 * mag + half * (np.abs(ref) + c * 2.0 ** -24 * mag) + 1e-36
    over = np.abs(got.detach().double().cpu().numpy() - ref) / tol
    print(f"    {name}: worst error {float(over.max()):.2f} of the bar", flush=True)
    assert np.isfinite(over).all() and over.max() <= 1.0, name


@KINDS
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 33, 64])
def test_few_channels_without_beta(D, dtype, gate):
    gdn = _gdn()
    gen = torch.Generator().manual_seed(D)
    lens = [5, 1700, 0, 3, 260, 1]
    T, N = sum(lens), len(lens)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    cu = torch.tensor(np.cumsum([0] + lens), dtype=I32, device=DEV)
    x, dy = randn(1, T, D).to(dtype).to(DEV), randn(1, T, D).to(dtype).to(DEV)
    g = (-torch.nn.functional.softplus(randn(1, T, D)) * torch.exp(torch.rand(D, generator=gen) * 6 - 6)).to(gate).to(DEV)
    h0, dht = randn(N, D).to(DEV), randn(N, D).to(DEV)
    y, f = gdn.gated_linear_recurrence(x, g, initial_state=h0, cu_seqlens=cu)
    ref, fin, mag, mfin = orc.scan(x, g, None, h0, cu)
    _near("y", y, ref, mag, 5)
    _near("final", f, fin, mfin, 5)
    y8 = gdn.checkpoint_activation(y)
    for kept, value in ((y, y), (y8, torch.from_numpy(orc.restore(*y8)))):
        got = gdn.gated_linear_recurrence_bwd(None, g, kept, dy, dht=dht, initial_state=h0, cu_seqlens=cu, output_dinitial=True)
        grads = orc.scan_bwd(None, g, value, dy, None, dht, h0, cu)
        assert got[2] is None
        for t, k in ((got[0], "dx"), (got[1], "dg"), (got[3], "dinitial")):
            _near(k, t, *grads[k], 8)
    for pdt in (F32, BF):
        pool, idx = randn(N + 2, D).to(pdt).to(DEV), torch.randperm(N + 2, generator=gen)[:N].to(I32)
        few = torch.tensor([0, 2, 3, 3, 7, 8, 9], dtype=I32, device=DEV)
        ref, after, mag, mafter = orc.scan_steps(x[:, :9], g[:, :9], pool, idx, None, None, few)
        y = gdn.gated_linear_recurrence_steps(x[:, :9], g[:, :9], pool, idx.to(DEV), cu_seqlens=few)
        _near("steps", y, ref, mag, 5)
        _near("pool", pool, after, mafter, 5)
