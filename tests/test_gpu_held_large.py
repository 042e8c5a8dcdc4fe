"""Values held in 8 and 4 bits in large passes: several parts a thread, through the cache and
past it, rows in any order with skipped ones.  Codes, scales and restored values are
equal to the float64 definition's, row by row of a sample; the whole tensors to what
calls on a few rows at a time make of them."""
import numpy as np
import pytest
import torch

from oracle import layer
from oracle import scan as orc

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
PAST = (256 << 20) + (1 << 22)   # bytes: more than passes through the cache have


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _np(t):
    return t.detach().double().cpu().numpy()


def _values(rows, D, extra, dtype, gen):
    """Rows whose sizes differ, with groups of zeros, infinities and NaNs among them."""
    wide = torch.randn(rows, D + extra, device=DEV, generator=gen).mul_(
        torch.exp(torch.randn(rows, 1, device=DEV, generator=gen) * 5)).to(dtype)
    v = wide[:, extra:]
    v[7::97, :min(D, 32)] = 0
    v[11::1009, D // 2] = float("nan")
    v[13::2003, D - 1] = float("inf")
    return v


def _near(name, got, ref, mag, c):
    """Within c roundings of the magnitude mag and that to the output's type."""
    half = torch.finfo(got.dtype).eps / 2
    tol = c * 2.0 ** -24 * mag + half * (np.abs(ref) + c * 2.0 ** -24 * mag) + 1e-36
    over = np.abs(_np(got) - ref) / tol
    print(f"    {name}: worst error {float(over.max()):.2f} of the bar", flush=True)
    assert np.isfinite(over).all() and over.max() <= 1.0, name


def _same(got, want):
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def _sample(rows, gen):
    return sorted({0, 1, 7, 11, 13, rows // 2, rows - 2, rows - 1} | set(torch.randint(0, rows, (150,), generator=gen).tolist()))


# values a row, extra columns of the rows, whether the pass is more than the cache holds: rows that share a workgroup
ROWS = [(33, 0, False), (33, 0, True), (129, 3, True), (100, 0, True), (1000, 8, True), (48, 0, True), (187, 0, False), (513, 1, True),
        (64, 5, True), (7, 0, True)]


@TYPES
@pytest.mark.parametrize("D,extra,past", ROWS)
def test_checkpoints_of_many_short_rows(D, extra, past, dtype):
    gdn = _gdn()
    gen, cgen = torch.Generator(device=DEV).manual_seed(D), torch.Generator().manual_seed(D)
    rows = (PAST if past else 100 << 20) // (D * (torch.finfo(dtype).bits // 8 + 1)) + 3
    x = _values(rows, D, extra, dtype, gen)
    c = gdn.checkpoint_activation(x)
    back = gdn.restore_activation(c, dtype)
    torch.cuda.synchronize()
    at = _sample(rows, cgen)
    codes, scales = orc.hold(x[at].cpu())
    assert (c.codes[at].cpu().numpy() == codes).all()
    np.testing.assert_array_equal(_np(c.scales[at]), scales)
    assert _same(back[at].cpu(), torch.from_numpy(orc.restore(codes, scales)).to(F32).to(dtype))
    # every row: parts of 100,003 rows, which take another launch
    for lo in range(0, rows, 100_003):
        part = slice(lo, min(lo + 100_003, rows))
        few = gdn.checkpoint_activation(x[part])
        assert torch.equal(few.codes, c.codes[part]) and torch.equal(few.scales.view(torch.int16), c.scales[part].view(torch.int16))
        assert _same(gdn.restore_activation(few, dtype), back[part])


def _cache_round(gdn, pool, slots, bits, gen, cgen):
    """The pool's slots to a cache in another order and back in a third, every eleventh pair skipped; checked on a sample
    against the definition, and that nothing else is written."""
    P, E = pool.shape[0], pool[0].numel()
    codes, scales = gdn.make_state_cache(pool, slots, bits)
    codes.fill_(85)
    src = torch.randperm(P, device=DEV, generator=gen).to(I32)
    at = torch.randperm(slots, device=DEV, generator=gen)[:P].to(I32)
    skip = torch.zeros(P, dtype=torch.bool, device=DEV)
    skip[3::11] = True
    w_src = torch.where(skip, torch.full_like(src, -1), src)
    gdn.state_cache_write(pool, w_src, codes, scales, at)
    torch.cuda.synchronize()
    unwritten = torch.ones(slots, dtype=torch.bool, device=DEV)
    unwritten[at[~skip].long()] = False
    assert (codes[unwritten] == 85).all() and not scales[unwritten].any()
    dst = torch.randperm(P, device=DEV, generator=gen).to(I32)
    other = torch.full_like(pool, 9.0)
    gdn.state_cache_read(codes, scales, torch.where(skip, torch.full_like(at, slots), at), other, dst)
    torch.cuda.synchronize()
    left = torch.ones(P, dtype=torch.bool, device=DEV)
    left[dst[~skip].long()] = False
    assert (other[left] == 9.0).all()
    for i in _sample(P, cgen)[::20 if E > 100_000 else 1]:
        if skip[i]:
            continue
        want_c, want_s = orc.hold(pool[int(src[i])].reshape(1, E).cpu(), bits)
        got_c = codes[int(at[i])].cpu().numpy()
        assert (got_c == (want_c if bits == 8 else orc.pack4(want_c))[0]).all(), i
        np.testing.assert_array_equal(_np(scales[int(at[i])]), want_s[0])
        want = torch.from_numpy(orc.restore(want_c, want_s)).to(F32).to(pool.dtype)[0]
        assert _same(other[int(dst[i])].reshape(E).cpu(), want), i


@TYPES
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,past", [(33, False), (48, True), (129, True), (1000, True), (1000, False), (7, True)])
def test_caches_of_many_short_states(D, past, bits, dtype):
    gdn = _gdn()
    gen, cgen = torch.Generator(device=DEV).manual_seed(D), torch.Generator().manual_seed(D)
    P = (PAST if past else 100 << 20) // int(D * (torch.finfo(dtype).bits // 8 + bits / 8)) + 5
    _cache_round(gdn, _values(P, D, 0, dtype, gen), P + 100, bits, gen, cgen)


# slots, elements a slot, whether the pass is more than the cache holds: long rows, four parts a thread, some with tails
LONG = [(1700, 10_001, False), (11_000, 10_001, True), (256, 1 << 19, True), (3000, 8192, False), (40, 500_003, False)]


@TYPES
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("P,E,past", LONG)
def test_caches_of_many_long_states(P, E, past, bits, dtype):
    gdn = _gdn()
    gen, cgen = torch.Generator(device=DEV).manual_seed(E), torch.Generator().manual_seed(E)
    nbytes = P * E * (torch.finfo(dtype).bits / 8 + bits / 8)
    assert P * -(-E // 8192) >= 2048 and (nbytes > 256 << 20) == past
    _cache_round(gdn, _values(P, E, 0, dtype, gen), P + 3, bits, gen, cgen)


@TYPES
@pytest.mark.parametrize("D", [32, 96, 128, 8224])
@pytest.mark.parametrize("past", [False, True], ids=["cached", "streamed"])
def test_checkpoints_of_rows_that_follow_each_other(past, D, dtype):
    gdn = _gdn()
    gen, cgen = torch.Generator(device=DEV).manual_seed(D), torch.Generator().manual_seed(D)
    rows = (PAST if past else 120 << 20) // (D * (torch.finfo(dtype).bits // 8 + 1)) + 3
    x = _values(rows, D, 0, dtype, gen)
    c = gdn.checkpoint_activation(x)
    back = gdn.restore_activation(c, dtype)
    at = _sample(rows, cgen)
    codes, scales = orc.hold(x[at].cpu())
    assert (c.codes[at].cpu().numpy() == codes).all()
    np.testing.assert_array_equal(_np(c.scales[at]), scales)
    assert _same(back[at].cpu(), torch.from_numpy(orc.restore(codes, scales)).to(F32).to(dtype))
    step = 20_003 * 128 // D + 1                       # the others: calls of a part a thread
    for lo in range(0, rows, step):
        few = gdn.checkpoint_activation(x[lo:lo + step])
        assert torch.equal(few.codes, c.codes[lo:lo + step])
        assert torch.equal(few.scales.view(torch.int16), c.scales[lo:lo + step].view(torch.int16))
        assert _same(gdn.restore_activation(few, dtype), back[lo:lo + step])


@TYPES
@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 24, 33, 64, 65, 100, 127, 128, 129, 187, 256, 300, 512, 520, 777, 1000, 1021, 1024])
def test_norm_gives_the_bits_of_the_norm_that_keeps_nothing(D, dtype):
    gdn = _gdn()
    gen = torch.Generator(device=DEV).manual_seed(D)
    for rows in (1, 300, 5000):
        x, z, w = (torch.randn(*s, device=DEV, generator=gen).to(dtype) for s in ((rows, D), (rows, D), (D,)))
        assert torch.equal(gdn.fused_gated_rms_norm_checkpoint(x, z, w)[0], gdn.fused_gated_rms_norm(x, z, w)), rows


# rows, values a row: forward and backward over several turns of several workgroups, in the cache and past it
NORMS = [(140_000, 128, BF), (530_001, 128, BF), (140_001, 128, F32), (300_000, 64, BF), (70_000, 256, BF), (33_001, 1024, BF),
         (17_003, 777, BF), (33_001, 777, F32), (400_003, 100, BF), (600_000, 100, BF), (66_000, 500, F32), (1_200_000, 33, BF),
         (140_003, 256, BF), (70_000, 500, BF), (90_000, 200, F32), (300_000, 60, F32)]


@pytest.mark.parametrize("rows,D,dtype", NORMS)
def test_norm_of_many_rows(rows, D, dtype):
    """y the bits of the norm that keeps nothing, codes the bits of checkpoint_activation; gradients of a sample of rows
    against the definition, dweight against its sum in 64 bits: at most 40 turns of a lane group, 64 groups and 512 rows of
    partial sums by 16 lanes add under 256 roundings to each term's own."""
    gdn = _gdn()
    gen, cgen = torch.Generator(device=DEV).manual_seed(rows), torch.Generator().manual_seed(rows)
    draw = lambda *s: torch.randn(*s, device=DEV, generator=gen).to(dtype)  # noqa: E731
    x, z, dy, w = draw(rows, D), draw(rows, D), draw(rows, D), draw(D)
    y, cx, cz = gdn.fused_gated_rms_norm_checkpoint(x, z, w)
    assert torch.equal(y, gdn.fused_gated_rms_norm(x, z, w))
    for c, v in ((cx, x), (cz, z)):
        e = gdn.checkpoint_activation(v)
        assert torch.equal(c.codes, e.codes) and torch.equal(c.scales, e.scales)
    dx, dz, dweight = gdn.fused_gated_rms_norm_checkpoint_bwd(cx, cz, w, dy)
    at = _sample(rows, cgen)
    xr, zr = (torch.from_numpy(orc.restore(_np(c.codes[at]), _np(c.scales[at]))) for c in (cx, cz))
    grads = layer.gated_norm_bwd(xr, zr, w, dy[at])
    _near("dx", dx[at], *grads["dx"], 128)
    _near("dz", dz[at], *grads["dz"], 128)
    ref, mag = torch.zeros(D, device=DEV, dtype=torch.float64), torch.zeros(D, device=DEV, dtype=torch.float64)
    for lo in range(0, rows, 50_000):
        s = slice(lo, min(lo + 50_000, rows))
        xv, zv = (gdn.restore_activation(gdn.Checkpoint(c.codes[s].contiguous(), c.scales[s].contiguous()), F32).double()
                  for c in (cx, cz))
        t = dy[s].double() * zv / (1 + torch.exp(-zv)) * xv * torch.rsqrt((xv * xv).mean(-1, keepdim=True) + 1e-6)
        ref += t.sum(0)
        mag += t.abs().sum(0)
    _near("dweight", dweight, _np(ref), _np(mag), 256)
    again = gdn.fused_gated_rms_norm_checkpoint_bwd(cx, cz, w, dy)
    assert all(torch.equal(a, b) for a, b in zip((dx, dz, dweight), again))
