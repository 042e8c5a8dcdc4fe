"""GPU parity of values held in 8 and 4 bits with the float64 definitions in
oracle/scan.py: codes and scales are equal, whatever the values; restored values are
code * scale, rounded once.  The gated norm that keeps its inputs gives the bits of
the norm that does not; its gradients have the bars of that norm's (128 and 256
roundings, see the norms' tests), at the values that the checkpoints stand for.
"""
import sys

import numpy as np
import pytest
import torch

from oracle import layer
from oracle import scan as orc

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -24
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(name, got, ref, mag, c):
    half = torch.finfo(got.dtype).eps / 2
    tol = c * ULP * mag + half * (np.abs(ref) + c * ULP * mag) + 1e-36
    g = _np(got)
    assert g.shape == ref.shape and np.isfinite(g).all(), name
    over = np.abs(g - ref) / tol
    worst = float(over.max()) if over.size else 0.0
    _say(f"    {name}: worst error {worst:.2f} of the bar")
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bar"


def _values(rows, D, dtype, seed):
    """Rows of all sizes, with ties, equal magnitudes, zeros, tiny groups, infinities and NaNs among them."""
    gen = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, D, generator=gen) * torch.exp(torch.randn(rows, 1, generator=gen) * 15)
    for i in range(rows):
        kind = i % 8
        if kind == 1:      # multiples of half a step below 127 or 7 steps
            v[i] = torch.randint(-254, 255, (D,), generator=gen) * 0.5
            v[i, ::32] = 127.0
        elif kind == 2:
            v[i] = torch.randint(-14, 15, (D,), generator=gen) * 0.5
            v[i, ::32] = 7.0
        elif kind == 3:    # a hair beside the ties
            v[i] = (torch.randint(-126, 127, (D,), generator=gen) + 0.5) * (1 + torch.randint(-1, 2, (D,), generator=gen) * 2.0 ** -23)
            v[i, ::32] = 127.0
        elif kind == 4:
            v[i] = torch.sign(v[i]) * v[i, 0].abs()
        elif kind == 5:
            v[i] = 0.0
        elif kind == 6:    # around the smallest group that is kept, and the largest numbers
            v[i] = v[i].sign() * 2.0 ** -100 * torch.rand(D, generator=gen) * (2 if i % 16 < 8 else 0.9)
            if i % 16 < 8:
                v[i, 0] = 3.3e38
    if rows > 20:
        v[9, D // 2], v[17, 0], v[18 % rows, D - 1] = float("nan"), float("inf"), -float("inf")
    return v.to(dtype)


@TYPES
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (40, 32), (40, 33), (30, 64), (25, 100), (24, 128), (64, 1001),
                                    (33, 2048), (21, 2049), (24, 4096), (70, 3)])
def test_checkpoint_is_the_definition(rows, D, dtype):
    gdn = _gdn()
    v = _values(rows, D, dtype, rows + D)
    codes, scales = orc.hold(v)
    c = gdn.checkpoint_activation(v.to(DEV))
    torch.cuda.synchronize()
    assert c.codes.shape == v.shape and (c.codes.cpu().numpy() == codes).all()
    np.testing.assert_array_equal(_np(c.scales), scales)
    for dt in (BF, F32):
        back = gdn.restore_activation(c, dt)
        want = torch.from_numpy(orc.restore(codes, scales)).to(F32).to(dt)
        assert back.dtype == dt and torch.equal(back.cpu().isnan(), want.isnan())
        assert torch.equal(back.cpu().nan_to_num(7.0), want.nan_to_num(7.0))
    # rows that are parts of wider ones, and that begin off alignment
    wide = torch.zeros(rows, D + 5, dtype=dtype, device=DEV)
    wide[:, 3:D + 3] = v.to(DEV)
    for part in (wide[:, 3:D + 3], torch.cat([v.new_zeros(1), v.flatten()]).to(DEV)[1:].view(rows, D)):
        again = gdn.checkpoint_activation(part)
        assert torch.equal(again.codes, c.codes) and torch.equal(again.scales.view(torch.int16), c.scales.view(torch.int16))


@TYPES
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("shape", [(2, 64, 64), (1, 1, 1), (3, 5), (40, 3), (701, 1), (4, 128, 128), (2051,)])
def test_state_cache(shape, bits, dtype):
    gdn = _gdn()
    P, C, n = 26, 25, 24
    E = int(np.prod(shape))
    v = _values(P, E, dtype, E + bits)
    gen = torch.Generator().manual_seed(E)
    pool = v.view(P, *shape).to(DEV)
    src, at = (torch.randperm(m, generator=gen)[:n].to(torch.int32) for m in (P, C))
    src[3], at[5], src[6] = -1, C, P
    ok = ((src >= 0) & (src < P) & (at < C)).numpy()
    codes, scales = gdn.make_state_cache(pool, C, bits)
    codes.fill_(85)
    scales.fill_(3.0)
    before_c, before_s = codes.clone(), scales.clone()
    gdn.state_cache_write(pool, src.to(DEV), codes, scales, at.to(DEV))
    want_c, want_s = orc.hold(v, bits)
    if bits == 4:
        want_c = orc.pack4(want_c)
    exp_c, exp_s = before_c.cpu().numpy().copy(), _np(before_s)
    for i in np.flatnonzero(ok):
        exp_c[at[i]], exp_s[at[i]] = want_c[src[i]], want_s[src[i]]
    assert (codes.cpu().numpy() == exp_c).all()
    np.testing.assert_array_equal(_np(scales), exp_s)
    # back into other slots, pairs outside skipped
    dst = torch.randperm(P, generator=gen)[:n].to(torch.int32)
    dst[0] = P + 3
    for dt in (BF, F32):
        other = torch.full((P, *shape), 9.0, dtype=dt, device=DEV)
        gdn.state_cache_read(codes, scales, at.to(DEV), other, dst.to(DEV))
        exp = torch.full((P, E), 9.0, dtype=dt)
        held_c, held_s = orc.hold(v, bits)
        for i in range(n):
            if at[i] < C and dst[i] < P:
                if ok[i]:
                    val = torch.from_numpy(orc.restore(held_c[src[i]], held_s[src[i]])).to(F32).to(dt)
                else:      # a cache slot that was not written holds what it held
                    c = before_c[at[i]].cpu().numpy().astype(np.int64)
                    if bits == 4:
                        c = np.stack([c & 15, c >> 4], -1).reshape(-1)[:E]
                        c = c - 16 * (c > 7)
                    val = torch.from_numpy(3.0 * c).to(dt)
                exp[dst[i]] = val
        got = other.cpu().view(P, E)
        assert torch.equal(got.isnan(), exp.isnan()) and torch.equal(got.nan_to_num(7.0), exp.nan_to_num(7.0))


def test_state_cache_slot_beyond_32_bits():
    """A cache and a pool of more than 2^31 elements: the last slots are written and read."""
    gdn = _gdn()
    E = 32 * 128 * 128
    P = (1 << 31) // E + 2
    one = torch.randn(1, 32, 128, 128, device=DEV, dtype=BF)
    pool = torch.zeros(P, 32, 128, 128, device=DEV, dtype=BF)
    pool[P - 1] = one[0]
    codes, scales = gdn.make_state_cache(pool, P)
    last, zero = (torch.tensor([i], dtype=torch.int32, device=DEV) for i in (P - 1, 0))
    gdn.state_cache_write(pool, last, codes, scales, last)
    c1, s1 = gdn.make_state_cache(one, 1)
    gdn.state_cache_write(one, zero, c1, s1, zero)
    assert torch.equal(codes[P - 1], c1[0]) and torch.equal(scales[P - 1], s1[0]) and not codes[:P - 1].any()
    pool.zero_()
    gdn.state_cache_read(codes, scales, last, pool, last)
    back = torch.empty_like(one)
    gdn.state_cache_read(c1, s1, zero, back, zero)
    assert torch.equal(pool[P - 1], back[0]) and not pool[:P - 1].any()


@TYPES
@pytest.mark.parametrize("rows,D", [(540_000, 7), (270_000, 33), (66_000, 100), (40_000, 1000), (20_000, 1001), (70_000, 1002)])
def test_many_short_rows(rows, D, dtype):
    """Rows that share a workgroup, several a thread: each is what a call on a few rows makes of it."""
    gdn = _gdn()
    gen = torch.Generator(device=DEV).manual_seed(rows)
    wide = torch.randn(rows, D + 3, device=DEV, generator=gen, dtype=F32).to(dtype)
    x = wide[:, 2:D + 2]
    c = gdn.checkpoint_activation(x)
    back = gdn.restore_activation(c, dtype)
    for at in (0, 255, rows // 3, rows - 1000, rows - 7):
        few = slice(at, min(at + 300, rows))
        codes, scales = orc.hold(x[few].cpu())
        assert (c.codes[few].cpu().numpy() == codes).all() and (_np(c.scales[few]) == scales).all()
        assert torch.equal(back[few].cpu(), torch.from_numpy(orc.restore(codes, scales)).to(F32).to(dtype))
    # the same through a pool's slots in another order, with pairs that are skipped, to 4 bits
    pool = x.contiguous()
    codes, scales = gdn.make_state_cache(pool, rows, 4)
    perm = torch.randperm(rows, device=DEV, generator=gen).to(torch.int32)
    src = torch.arange(rows, device=DEV, dtype=torch.int32)
    src[5::11] = -1
    gdn.state_cache_write(pool, src, codes, scales, perm)
    other = torch.full_like(pool, 9.0)
    gdn.state_cache_read(codes, scales, perm, other, src)
    assert (other[5::11] == 9.0).all() and not codes[perm[5::11].long()].any()
    for at in (0, rows // 2, rows - 300):
        held = orc.hold(pool[at:at + 300].cpu(), 4)
        want = torch.from_numpy(orc.restore(*held)).to(F32).to(dtype)
        keep = src[at:at + 300].cpu() >= 0
        assert torch.equal(other[at:at + 300].cpu()[keep], want[keep])


def test_more_rows_than_a_launch_has_workgroups():
    """2^24 + 3 rows of a head: rows that follow each other are one."""
    gdn = _gdn()
    n = (1 << 24) + 3
    x = torch.randn(n, 128, device=DEV, dtype=BF)
    c = gdn.checkpoint_activation(x)
    back = gdn.restore_activation(c)
    for at in (0, 1 << 20, n - 200):
        codes, scales = orc.hold(x[at:at + 200].cpu())
        assert (c.codes[at:at + 200].cpu().numpy() == codes).all() and (_np(c.scales[at:at + 200]) == scales).all()
        assert torch.equal(back[at:at + 200].cpu(), torch.from_numpy(orc.restore(codes, scales)).to(F32).to(BF))


NORMS = [((5, 4), 128), ((3, 1, 6), 64), ((7,), 1), ((2, 3), 100), ((9, 2), 129), ((3,), 512), ((2, 2), 777),
         ((2,), 1024), ((300, 32), 128), ((3, 5), 1021), ((700, 9), 5), ((90, 10), 187), ((70, 3), 9), ((500, 7), 96),
         ((32,), 128), ((8, 8), 128), ((65,), 128), ((17,), 512)]   # one workgroup's turns, and one row more


@TYPES
@pytest.mark.parametrize("lead,D", NORMS)
def test_norm_that_keeps_its_inputs(lead, D, dtype):
    gdn = _gdn()
    gen = torch.Generator().manual_seed(D)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, dy, w = randn(*lead, D).to(dtype).to(DEV), randn(*lead, D).to(dtype).to(DEV), (randn(D) * 0.3 + 1).to(dtype).to(DEV)
    heads = lead[-1] if len(lead) > 1 else 1
    wide = (randn(*lead[:-1] if heads > 1 else lead, heads * D + 5) * 2).to(dtype).to(DEV)
    z = wide[..., 5:].view(*lead, D)
    _say(f"[norm, inputs in 8 bits] {lead} {D} {dtype}")
    ref, mag = layer.gated_norm(x, z, w)
    y, cx, cz = gdn.fused_gated_rms_norm_checkpoint(x, z, w)
    torch.cuda.synchronize()
    _near("y", y, ref, mag, 64)
    for c, v in ((cx, x), (cz, z)):
        codes, scales = orc.hold(v)
        assert (c.codes.cpu().numpy() == codes).all() and (_np(c.scales) == scales).all()
    got = gdn.fused_gated_rms_norm_checkpoint_bwd(cx, cz, w, dy)
    xr, zr = (torch.from_numpy(orc.restore(*c)) for c in (cx, cz))
    grads = layer.gated_norm_bwd(xr, zr, w, dy)
    for t, name, c in zip(got, ("dx", "dz", "dweight"), (128, 128, 256)):
        _near(name, t, *grads[name], c)
    assert got[0].dtype == dtype and got[2].dtype == F32
    again = gdn.fused_gated_rms_norm_checkpoint_bwd(cx, cz, w.float(), dy)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
