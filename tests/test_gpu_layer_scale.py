"""GPU parity of the short convolution and the RMS norms at the sizes whose
launches differ from small ones: strips of several load batches up to the longest,
waves that walk several rows, passes that are streamed past the last cache, and
the wide form of the column sums.  Compared on the device with the whole-tensor
float64 forms of oracle/layer_whole.py.

Bars, as for the small sizes: an output x of magnitude m is off by at most
c 2^-24 m + half (|x| + c 2^-24 m), half = eps/2 of its type, with c the number of
fp32 roundings on the longest path:
  conv 8 (W products and the bias, the exponential, the reciprocal, the product);
  its gradients 16; weights' gradients 16 + the tokens of a strip + 2 for its
  workgroup's four strips + the column sum's groups per row lane and its tree (6);
  norms 64 (16 squares a lane, 22 to add the group, the mean, the root, products),
  their gradients 128 (two such sums), weights' 64 + the rows that a group walks +
  the groups of a workgroup (32 at most) + at most 64 workgroups a row lane + 6.
Histories are equal bit for bit.
"""
import random
import sys

import pytest
import torch

from oracle import layer_whole

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -24
LAST_CACHE = 256 << 20
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _near(name, got, ref, mag, c):
    assert got.numel() == ref.numel(), (name, got.shape, ref.shape)
    half = torch.finfo(got.dtype).eps / 2
    g, ref, mag = got.reshape(-1).double(), ref.reshape(-1), mag.reshape(-1)
    assert bool(torch.isfinite(g).all()), f"{name}: not finite"
    over = (g - ref).abs() / (c * ULP * mag + half * (ref.abs() + c * ULP * mag) + 1e-36)
    worst = float(over.max())
    _say(f"    {name}: worst error {worst:.2f} of the bar")
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bar at element {int(over.argmax())} of {list(got.shape)}"


class Draw:
    def __init__(self, seed):
        self.gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(self, *shape, std=1.0, dtype=F32):
        return (torch.randn(*shape, generator=self.gen, device=DEV) * std).to(dtype)


# ---------------------------------------------------------------------------
# Short convolution
# ---------------------------------------------------------------------------
def _strip(T, D, cols, batch, most):
    """Tokens of a strip: `most`, halved down to one load batch while there are fewer than 2048 waves."""
    waves = lambda L: -(-T // L) * -(-D // (64 * cols))
    L = most
    while L > batch and waves(L) < 2048:
        L //= 2
    return L


def _lens(T, seed):
    """Ragged lengths that sum to T: empty and single tokens, ends inside and at the ends of load batches (3 and 4
    tokens) and strips (12, 16, 48, 64), sequences over many strips."""
    r, lens = random.Random(seed), []
    pick = [0, 0, 1, 1, 2, 3, 4, 5, 11, 12, 13, 16, 24, 31, 47, 48, 49, 64, 65, 100, 301, 603]
    while sum(lens) < T:
        lens.append(min(r.choice(pick), T - sum(lens)))
    return lens + [0]


CONV = {   # W, tokens, pieces, rows of x beyond them, (strip forward, backward), equal rows (or ragged), bias, SiLU
    "w4_12_48": (4, 3001, (2051, 2049, 4100), 3, (12, 48), 0, True, True),
    "w4_12_24": (4, 1500, (2050, 2050, 4100), 0, (12, 24), 0, False, True),
    "w4_6_12": (4, 1501, (1100, 1100, 2200), 5, (6, 12), 0, True, True),
    "w4_3_6": (4, 500, (8200,), 0, (3, 6), 5, False, False),
    "w3_16_64": (3, 4001, (2051, 2049, 4100), 1, (16, 64), 0, True, True),
    "w3_16_32": (3, 2002, (8200,), 0, (16, 32), 2, False, True),
    "w2_16_64": (2, 4004, (2051, 2049, 4100), 7, (16, 64), 4, True, True),
    "w2_8_16": (2, 1001, (2050, 2050, 4100), 0, (8, 16), 0, False, False),
    "w2_4_8": (2, 501, (8200,), 2, (4, 8), 0, True, True),
    # more than the last cache holds: streamed
    "stream_w4": (4, 8300, (2048, 2048, 4096), 4096, (12, 48), 0, True, True),
    "stream_w4_odd": (4, 8300, (2051, 2049, 4100), 1, (12, 48), 0, False, True),
    "stream_w3": (3, 8300, (2048, 2048, 4096), 0, (16, 64), 0, False, True),
    "stream_w2": (2, 8300, (2048, 2048, 4096), 0, (16, 64), 0, True, True),
}


@TYPES
@pytest.mark.parametrize("name", list(CONV))
def test_conv_strips(name, dtype):
    gdn = _gdn()
    W, T, sizes, extra, strips, rows, bias, silu = CONV[name]
    D, batch = sum(sizes), 3 if W == 4 else 4
    fwd, bwd = _strip(T, D, 8, batch, 4 * batch), _strip(T, D, 4, batch, 16 * batch)
    assert (fwd, bwd) == strips
    if name.startswith("stream"):
        assert T * D * dtype.itemsize * 2 > LAST_CACHE
    _say(f"[conv strips] {name} {dtype}")
    d = Draw(sum(map(ord, name)))
    B = max(rows, 1)
    lens = [T // rows] * rows if rows else _lens(T, W)
    assert sum(lens) == T
    cu = None if rows else torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV)
    x = d.randn(B, T // B, D + extra, dtype=dtype)[..., extra:]
    w, b = d.randn(D, W, std=0.5, dtype=dtype), d.randn(D, std=0.2, dtype=dtype) if bias else None
    h0 = d.randn(len(lens), D, W - 1, dtype=dtype)
    kw = dict(cu_seqlens=cu, activation="silu" if silu else None)
    # forward
    ref, fin, mag = layer_whole.conv(x, w, b, h0, lens, silu)
    y, final = gdn.causal_conv1d(x, w, b, initial_state=h0, split_sizes=sizes, **kw)
    torch.cuda.synchronize()
    _near("y", torch.cat(y, -1), ref, mag, 8)
    assert bool((final.double() == fin).all())
    h = h0.clone()
    y2, _ = gdn.causal_conv1d(x, w, b, initial_state=h, final_state=h, split_sizes=sizes, **kw)
    assert torch.equal(h, final) and all(torch.equal(a, c) for a, c in zip(y, y2))
    del ref, mag, y, y2
    # backward
    dy = [d.randn(B, T // B, n, dtype=dtype) for n in sizes]
    shape = gdn.gdn_conv_shape(B, T // B, D, W, len(lens), 0 if dtype == BF else 1, 0 if dtype == BF else 1, D + extra)
    groups = -(-(-(-T // bwd)) // 4)
    assert gdn.gdn_conv_bwd_workspace_bytes(shape) == groups * (W + 1) * D * 4     # the strip is the one named above
    call = lambda: gdn.causal_conv1d_bwd(x, w, dy, b, initial_state=h0, output_dinitial=True, **kw)
    got = call()
    torch.cuda.synchronize()
    ref = layer_whole.conv_bwd(x, w, torch.cat(dy, -1), b, h0, lens, silu)
    sums = 16 + bwd + 2 + -(-groups // (64 if (W + 1) * D <= 8192 else 4)) + 6
    for t, part, c in zip(got, ("dx", "dweight", "dbias", "dinitial"), (16, sums, sums, 16)):
        if t is not None:
            _near(part, t, *ref[part], c)
    assert all(a is c is None or torch.equal(a, c) for a, c in zip(got, call()))


# ---------------------------------------------------------------------------
# RMS norms
# ---------------------------------------------------------------------------
@TYPES
@pytest.mark.parametrize("rows,D", [
    # more rows than the forward launch has groups of lanes, for each size of a group
    (270001, 64), (140001, 128), (70003, 250), (40003, 512), (40001, 1021),
    # more than the last cache holds, rows of an odd and an even length
    (241001, 187), (45001, 1024)])
def test_gated_norm_rows(rows, D, dtype):
    gdn = _gdn()
    d = Draw(D)
    if rows in (241001, 45001):
        assert rows * D * 3 * dtype.itemsize > LAST_CACHE
    _say(f"[gated norm] {rows} x {D} {dtype}")
    x, dy, w = d.randn(rows, D, dtype=dtype), d.randn(rows, D, dtype=dtype), (d.randn(D, std=0.3) + 1).to(dtype)
    z = d.randn(rows, D + 3, std=2.0, dtype=dtype)[:, 3:]
    _near("y", gdn.fused_gated_rms_norm(x, z, w), *layer_whole.gated_norm(x, z, w), 64)
    got = gdn.fused_gated_rms_norm_bwd(x, z, w, dy)
    ref = layer_whole.gated_norm_bwd(x, z, w, dy)
    groups = 2048 * 64 // {64: 8, 128: 16, 250: 32, 187: 32}.get(D, 64)
    for t, part, c in zip(got, ("dx", "dz", "dweight"), (128, 128, 64 + -(-rows // groups) + 32 + 64 + 6)):
        _near(part, t, *ref[part], c)
    assert all(torch.equal(a, b) for a, b in zip(got, gdn.fused_gated_rms_norm_bwd(x, z, w, dy)))


@TYPES
@pytest.mark.parametrize("rows,D", [
    (270001, 64), (40001, 1021), (9001, 2041), (5003, 4096), (700, 8192), (300, 16384),
    # more than the last cache holds
    (33001, 2048), (9003, 4001), (7001, 5001), (3801, 9001)])
def test_add_norm_rows(rows, D, dtype):
    gdn = _gdn()
    d = Draw(D)
    if rows in (33001, 9003, 7001, 3801):
        assert rows * D * 4 * dtype.itemsize > LAST_CACHE
    _say(f"[add norm] {rows} x {D} {dtype}")
    x, res, dy, dh = (d.randn(rows, D, std=s, dtype=dtype) for s in (1.0, 2.0, 1.0, 1.0))
    w = d.randn(D, std=0.3, dtype=dtype)
    kw = dict(residual_scale=0.7, weight_offset=1.0)
    ref, h, mag, size = layer_whole.add_norm(x, res, w, **kw)
    y, hid = gdn.fused_add_rms_norm(x, res, w, **kw)
    _near("hidden", hid, h, size, 2)
    _near("y", y, ref, mag, 64)
    again = res.clone()
    y2, _ = gdn.fused_add_rms_norm(x, again, w, hidden=again, **kw)
    assert torch.equal(again, hid) and torch.equal(y2, y)
    del ref, h, mag, size, y, y2, again
    got = gdn.fused_add_rms_norm_bwd(dy, dh, hid, w, **kw)
    ref = layer_whole.add_norm_bwd(dy, dh, hid, w, **kw)
    groups = 2048 * 64 // (8 if D == 64 else 64 if D <= 1024 else 256 if D <= 2048 else 512 if D <= 4096 else 512)
    for t, part, c in zip(got, ("dx", "dresidual", "dweight"), (128, 128, 64 + -(-rows // groups) + 32 + 64 + 6)):
        _near(part, t, *ref[part], c)
    assert all(torch.equal(a, b) for a, b in zip(got, gdn.fused_add_rms_norm_bwd(dy, dh, hid, w, **kw)))
