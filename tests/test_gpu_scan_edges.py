"""The gated linear recurrence at the edges of its numbers: gates that are NaN in any of a
NaN's bit patterns, above zero, and over the whole range of the decays."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(seed, T, D, dtype=F32, gate=F32):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(1, T, D, generator=gen).to(dtype).to(DEV)
    g = (-torch.nn.functional.softplus(torch.randn(1, T, D, generator=gen)) * 0.2).to(gate).to(DEV)
    b = torch.rand(1, T, D, generator=gen).to(gate).to(DEV)
    return x, g, b, torch.randn(1, T, D, generator=gen).to(dtype).to(DEV)


def _cu(*lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=I32, device=DEV)


def _bits(pattern):
    """The fp32 number of these bits, as the int32 that they are."""
    return int(np.array(pattern, dtype=np.uint32).view(np.int32))


@pytest.mark.parametrize("D", [3, 37, 133])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_a_gate_that_is_not_a_number(dtype, D):
    """The states from a NaN gate on, and the gradients up to it, are NaNs whatever bits the NaN's payload has; other
    channels and sequences are the bits that they were."""
    gdn = _gdn()
    lens, at, ch = (40, 700, 30), 45, D // 2
    cu, T = _cu(*lens), sum(lens)
    x, g, b, dy = _inputs(D, T, D, dtype)

    def both(g):
        y, f = gdn.gated_linear_recurrence(x, g, b, cu_seqlens=cu)
        return (y, f, *gdn.gated_linear_recurrence_bwd(x, g, y, dy, b, cu_seqlens=cu, output_dinitial=True))

    clean = both(g)
    for pattern in (0x7fc00000, 0x7fffffff, 0xffffffff, 0x7fc00001, 0xffc001ff, 0x7f800001):
        bad = g.clone()
        bad.view(I32)[0, at, ch] = _bits(pattern)
        y, f, dx, dg, dbeta, dinitial = got = both(bad)
        assert y[0, at:740, ch].isnan().all() and f[1, ch].isnan(), hex(pattern)
        assert dx[0, 40:at, ch].isnan().all() and dg[0, 40:at + 1, ch].isnan().all() and dinitial[1, ch].isnan(), hex(pattern)
        for u, v in zip(got, clean):
            same = torch.ones_like(u, dtype=torch.bool)
            if u.dim() == 2:
                same[1, ch] = False
            else:
                same[0, 40:740, ch] = False
            assert torch.equal(u[same], v[same]), hex(pattern)
        # a token at a time
        pool, slots = torch.zeros(2, D, device=DEV), torch.tensor([1, 0], dtype=I32, device=DEV)
        ys = gdn.gated_linear_recurrence_steps(x[0, 44:48].view(2, 2, D), bad[0, 44:48].view(2, 2, D), pool, slots)
        assert ys[0, 1, ch].isnan() and pool[1, ch].isnan() and not ys[0, 0].isnan().any(), hex(pattern)
        ys[0, 1, ch], pool[1, ch] = 0, 0
        assert ys.isfinite().all() and pool.isfinite().all()


def test_a_gate_above_zero():
    """Not in the gates' range, but no other number than e^g: within its rounding below 88, infinite from 89 on."""
    gdn = _gdn()
    g = torch.tensor([1e-3, 0.5, 3.0, 40.0, 88.0, 89.0, 100.0, 1e4, 3e6, 1e10, 1e30], device=DEV).view(1, 1, -1)
    x, h = torch.zeros_like(g), torch.ones(1, g.shape[-1], device=DEV)
    y, f = gdn.gated_linear_recurrence(x, g, initial_state=h)
    assert torch.equal(y[:, 0], f) and (f[0, 5:] == float("inf")).all()
    np.testing.assert_allclose(_np(f)[0, :5], np.exp(_np(g)[0, 0, :5]), rtol=6 * 2.0 ** -24)


@pytest.mark.parametrize("gate", [F32, BF], ids=["fp32", "bf16"])
def test_the_decay_over_its_range(gate):
    """e^g alone (a state of one, no input) against float64, in units of 2^-24 of its value.  e^g = 2^n q(r), |r| <= 0.35:
    two roundings of r of at most 0.25 each, one of the last sum, q, of at most 0.8 (half a step of a number between 0.7 and
    1.42), one of the sum before it, which r carries into q, of at most 0.25, and 0.1 of the earlier ones and of the
    polynomial: 1.65 if all of them met, 1.32 in every 13th number of the range.  The recurrence's bars take 1.5 for it,
    and so does this one.  Below -87 it is 0."""
    gdn = _gdn()
    gen = torch.Generator().manual_seed(1)
    n = 1 << 18
    g = torch.cat([-torch.rand(n, generator=gen) * 87, -torch.exp(torch.rand(n, generator=gen) * 20 - 15.6).clamp(max=87),
                   torch.tensor([0.0, -0.0, -87.0, -1e-30])]).to(gate).to(DEV)
    g, D = g[g >= -87].view(1, 1, -1), int((g >= -87).sum())
    want = np.exp(_np(g).reshape(-1))
    one, zero, slot = torch.ones(1, D, device=DEV), torch.zeros(1, 1, D, device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    pool = one.clone()
    _, f = gdn.gated_linear_recurrence(zero.to(gate), g, initial_state=one)
    gdn.gated_linear_recurrence_steps(zero.to(gate), g, pool, slot)
    back = gdn.gated_linear_recurrence_bwd(None, g, zero.to(gate), zero.to(gate), dht=one, output_dinitial=True)[3]
    for name, t in (("forward", f), ("steps", pool), ("backward", back)):
        over = np.abs(_np(t).reshape(-1) - want) / want * 2.0 ** 24
        print(f"    {name}: worst {over.max():.3f} 2^-24 at g = {float(g.reshape(-1)[int(over.argmax())])}", flush=True)
        assert over.max() <= 1.5, name
    low = torch.tensor([-87.5, -88.0, -1e3, -1e30, torch.finfo(gate).min, -float("inf")], device=DEV).to(gate).view(1, 1, -1)
    assert not gdn.gated_linear_recurrence(torch.zeros_like(low), low, initial_state=one[:, :6])[1].any()


def test_a_million_sequences():
    """2^20 sequences of one token of 4096 channels each: from zero, y and the final states are x, and dx is dy."""
    gdn = _gdn()
    N, D = 1 << 20, 4096
    x = torch.randn(1, N, D, device=DEV, dtype=BF)
    g = torch.full((1, 1, 1), -0.5, device=DEV, dtype=BF).expand(1, N, D).contiguous()
    cu = torch.arange(N + 1, device=DEV, dtype=I32)
    y, f = gdn.gated_linear_recurrence(x, g, cu_seqlens=cu)
    assert torch.equal(y, x)
    assert torch.equal(f, x[0].float())
    del f
    dx, dg, _, _ = gdn.gated_linear_recurrence_bwd(None, g, y, x, cu_seqlens=cu)
    assert torch.equal(dx, x) and not dg.any()


@pytest.mark.parametrize("D", [2, 40, 133])
@pytest.mark.parametrize("dtype,gate", [(BF, F32), (BF, BF), (F32, F32)], ids=["bf16_fp32", "bf16", "fp32"])
def test_no_state_is_finite_behind_an_infinity(dtype, gate, D):
    """An infinite input, or one in the initial state, under decays whose product underflows within a strip of tokens, a
    tile, or not at all: every later state of the channel's sequence is an infinity or a NaN, with small decays the
    infinity; of gradients, every earlier one.  Other channels are the bits that they were."""
    gdn = _gdn()
    lens, at = (50, 5000, 30), 1700
    cu, T = _cu(*lens), sum(lens)
    x, _, b, dy = _inputs(D, T, D, dtype, gate)
    gen = torch.Generator().manual_seed(5)
    h0, dht = torch.randn(3, D, generator=gen).to(DEV), torch.randn(3, D, generator=gen).to(DEV)
    inf = float("inf")
    for rate in (1e-3, 0.5, 7.0, 60.0):
        g = (-(torch.rand(1, T, D, generator=gen) + 0.5) * rate).to(gate).to(DEV)

        def both(x, h0, dy, dht):
            y, f = gdn.gated_linear_recurrence(x, g, b, initial_state=h0, cu_seqlens=cu)
            return (y, f, *gdn.gated_linear_recurrence_bwd(x, g, y, dy, b, dht=dht, initial_state=h0, cu_seqlens=cu,
                                                           output_dinitial=True))

        clean = both(x, h0, dy, dht)
        bad = [t.clone() for t in (x, h0, dy, dht)]
        bad[0][0, at, 0] = -inf
        bad[2][0, at, 0] = inf
        bad[1][1, D - 1] = inf
        bad[3][1, D - 1] = inf
        got = both(*bad)
        y, f, dx, _, _, dinitial = got
        for t in (y[0, at:5050, 0], f[1, 0], y[0, 50:5050, D - 1], f[1, D - 1], dx[0, 50:at + 1, 0], dinitial[1, 0],
                  dx[0, 50:5050, D - 1], dinitial[1, D - 1]):
            assert not t.isfinite().any(), rate
        if rate < 0.01:   # 5000 tokens are e^-10: no product is zero
            assert (y[0, at:5050, 0] == -inf).all() and (y[0, 50:5050, D - 1] == inf).all()
            assert (dx[0, 50:at + 1, 0] == inf).all() and dinitial[1, D - 1] == inf
        for u, v in zip(got, clean):
            same = torch.ones_like(u, dtype=torch.bool)
            for ch in (0, D - 1):
                if u.dim() == 2:
                    same[1, ch] = False
                else:
                    same[0, 50:5050, ch] = False
            assert torch.equal(u[same], v[same]), rate
