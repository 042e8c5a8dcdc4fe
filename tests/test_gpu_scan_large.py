"""The gated linear recurrence in passes that are streamed past the cache, which large
batches take: the same bits as passes over a part of their channels, which are small
enough not to be streamed and are compared with the definition elsewhere (a channel's
arithmetic does not depend on the channels beside it); and the definition on slices
that a token that forgets everything cuts off."""
import numpy as np
import pytest
import torch

from oracle import scan as orc

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
D, PART = 512, 96        # rows of whole lines; parts of whole groups of 32, in bf16 not of whole lines
KINDS = pytest.mark.parametrize("dtype,gate", [(BF, F32), (BF, BF), (F32, F32)], ids=["bf16_fp32", "bf16", "fp32"])
BETA = pytest.mark.parametrize("with_beta", [True, False], ids=["beta", "no_beta"])


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(name, got, ref, mag, c):
    """The bar of the recurrence's other tests: c roundings of an fp32 evaluation, and that to the output's type."""
    half = torch.finfo(got.dtype).eps / 2
    tol = c * 2.0 ** -24 * mag + half * (np.abs(ref) + c * 2.0 ** -24 * mag) + 1e-36
    over = np.abs(_np(got) - ref) / tol
    print(f"    {name}: worst error {float(over.max()):.2f} of the bar", flush=True)
    assert np.isfinite(over).all() and over.max() <= 1.0, name


def _inputs(dtype, gate, with_beta, token):
    """A packed batch of a little more than 256 MiB at `token` bytes a token and channel."""
    T = (256 << 20) // (token * D) + 1500
    lens = [700, 0, 1, T // 2, 33]
    lens.append(T - sum(lens) - 5)
    gen = torch.Generator(device=DEV).manual_seed(T)
    draw = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    rate = torch.exp(torch.rand(D, device=DEV, generator=gen) * 7 - 7)
    g = (-rate * torch.nn.functional.softplus(draw(1, T, D))).to(gate)
    cuts = [1500, 1500 + T // 4, T - 900]               # slices of 600 tokens of one sequence before and behind them
    for at in cuts:
        g[:, at] = -1e30
    x = draw(1, T, 2 * D).to(dtype)[..., D:]
    beta = torch.rand(1, T, D, device=DEV, generator=gen).to(gate) if with_beta else None
    cu = torch.tensor(np.cumsum([0] + lens), dtype=I32, device=DEV)
    return x, g, beta, draw(len(lens), D), cu, draw(1, T, D).to(dtype), draw(len(lens), D), cuts


def _cols(t, c):
    return None if t is None else t[..., c]


PARTS = [slice(at, at + PART) for at in (0, 96, 192, 288, 384, 416)]


@BETA
@KINDS
def test_streamed_forward(dtype, gate, with_beta):
    gdn = _gdn()
    token = 2 * dtype.itemsize + (2 if with_beta else 1) * gate.itemsize
    x, g, b, h0, cu, _, _, cuts = _inputs(dtype, gate, with_beta, token)
    y, f = gdn.gated_linear_recurrence(x, g, b, initial_state=h0, cu_seqlens=cu)
    used = int(cu[-1])
    for c in PARTS:
        y1, f1 = gdn.gated_linear_recurrence(_cols(x, c), _cols(g, c), _cols(b, c), initial_state=h0[:, c], cu_seqlens=cu)
        assert torch.equal(y[:, :used, c], y1[:, :used]) and torch.equal(f[:, c], f1), c
    for at in cuts:
        s = slice(at, at + 600)
        ref, _, mag, _ = orc.scan(x[:, s], g[:, s], None if b is None else b[:, s])
        _near("y", y[:, s], ref, mag, 5)
    pool, slots = torch.cat([h0, h0[:1]]), torch.tensor([3, 6, 1, 0, 5, 2], dtype=I32, device=DEV)
    start = torch.empty_like(pool)
    start[slots.long()] = h0
    yp, _ = gdn.gated_linear_recurrence(x, g, b, cu_seqlens=cu, state_pool=start, state_indices=slots)
    assert torch.equal(yp[:, :used], y[:, :used]) and torch.equal(start[slots.long()], f)


@pytest.mark.parametrize("held", [False, True], ids=["tensors", "checkpoints"])
@BETA
@KINDS
def test_streamed_backward(dtype, gate, with_beta, held):
    gdn = _gdn()
    gates = 2 if with_beta else 1
    token = 2 * dtype.itemsize + 2 * gates * gate.itemsize + gates * (1 if held else dtype.itemsize)
    x, g, b, h0, cu, dy, dht, cuts = _inputs(dtype, gate, with_beta, token)
    y, _ = gdn.gated_linear_recurrence(x, g, b, initial_state=h0, cu_seqlens=cu)
    used = int(cu[-1])
    y[:, used:] = 0
    if held:
        x, y = gdn.checkpoint_activation(x), gdn.checkpoint_activation(y)

    def call(c):
        cut = lambda t: (gdn.Checkpoint(t.codes[..., c], t.scales[..., c.start // 32:-(-c.stop // 32)])  # noqa: E731
                         if held else t[..., c])
        return gdn.gated_linear_recurrence_bwd(cut(x) if with_beta else None, g[..., c], cut(y), dy[..., c], _cols(b, c),
                                               dht=dht[:, c], initial_state=h0[:, c], cu_seqlens=cu, output_dinitial=True)

    got = call(slice(0, D))
    for c in PARTS:
        for u, v in zip(got, call(c)):
            if u is not None:
                u, v = (u[..., c], v) if u.dim() == 2 else (u[:, :used, c], v[:, :used])
                assert torch.equal(u, v), c
    full = lambda t, s: torch.from_numpy(orc.restore(_np(t.codes[:, s]), _np(t.scales[:, s]))) if held else t[:, s]  # noqa: E731
    for at in cuts[:2]:
        # a gradient does not come out of the token after the slice, which forgets everything, and a state not into it
        s = slice(at - 600, at)
        ref = orc.scan_bwd(full(x, s) if with_beta else dy[:, s], g[:, s], full(y, s), dy[:, s], b[:, s] if with_beta else None)
        for t, k in zip(got, ("dx", "dg", "dbeta")):
            if t is not None:
                _near(k, t[:, s][:, 1:], *(r[:, 1:] for r in ref[k]), 8)
