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


@pytest.mark.parametrize("D", [1, 3, 8, 40, 64, 65])
def test_few_channels_of_far_rows(D):
    """Rows 2^22 elements apart, so that a strip's tokens are more than 2^32 bytes behind the first row: the bits of the call
    on their copies, forward and backward, with beta and without."""
    gdn = _gdn()
    T, far = 1100, 1 << 22
    gen = torch.Generator(device=DEV).manual_seed(D)
    wide = torch.zeros(1, T, far, device=DEV, dtype=BF)
    x, g, b = wide[..., 100:100 + D], wide[..., 1000:1000 + D], wide[..., far - D:]
    x.copy_(torch.randn(1, T, D, device=DEV, generator=gen))
    g.copy_(-torch.rand(1, T, D, device=DEV, generator=gen) * 0.2)
    b.copy_(torch.rand(1, T, D, device=DEV, generator=gen))
    dy, h0 = torch.randn(1, T, D, device=DEV, generator=gen).to(BF), torch.randn(1, D, device=DEV, generator=gen)
    for beta in (b, None):
        cut = [t if t is None else t.clone(memory_format=torch.contiguous_format) for t in (x, g, beta)]
        y, f = gdn.gated_linear_recurrence(x, g, beta, initial_state=h0)
        y1, f1 = gdn.gated_linear_recurrence(*cut, initial_state=h0)
        assert torch.equal(y, y1) and torch.equal(f, f1)
        one = gdn.gated_linear_recurrence_bwd(x, g, y, dy, beta, initial_state=h0, output_dinitial=True)
        two = gdn.gated_linear_recurrence_bwd(cut[0], cut[1], y, dy, cut[2], initial_state=h0, output_dinitial=True)
        assert all(u is v is None or torch.equal(u, v) for u, v in zip(one, two))


@pytest.mark.parametrize("D", [2, 8, 40, 64])
@KINDS
def test_few_channels_over_several_blocks_of_tiles(dtype, gate, D):
    """70,000 tokens of one sequence, behind and before short ones, without beta: gradients from tensors and from checkpoints."""
    gdn = _gdn()
    gen = torch.Generator().manual_seed(D)
    lens = [3, 70_000, 40]
    T = sum(lens)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=I32, device=DEV)
    y, dy = torch.randn(1, T, D, generator=gen).to(dtype).to(DEV), torch.randn(1, T, D, generator=gen).to(dtype).to(DEV)
    g = (-torch.nn.functional.softplus(torch.randn(1, T, D, generator=gen)) * torch.exp(torch.rand(D, generator=gen) * 6 - 8))
    g = g.to(gate).to(DEV)
    g[:, 60_000] = -1e30
    dht = torch.randn(3, D, generator=gen).to(DEV)
    y8 = gdn.checkpoint_activation(y)
    held = torch.from_numpy(orc.restore(*y8))
    ref = orc.scan_bwd(None, g, y, dy, None, dht, None, cu)
    got = gdn.gated_linear_recurrence_bwd(None, g, y, dy, dht=dht, cu_seqlens=cu, output_dinitial=True)
    _near("dx", got[0], *ref["dx"], 8)
    _near("dg", got[1], *ref["dg"], 8)
    _near("dinitial", got[3], *ref["dinitial"], 8)
    ref = orc.scan_bwd(None, g, held, dy, None, dht, None, cu)
    got = gdn.gated_linear_recurrence_bwd(None, g, y8, dy, dht=dht, cu_seqlens=cu)
    _near("dx, 8 bits", got[0], *ref["dx"], 8)
    _near("dg, 8 bits", got[1], *ref["dg"], 8)
