"""Pins of the float64 definitions in oracle/scan.py (no GPU): worked examples, the
convolution of impulses, central differences, and the format's own promises."""
import numpy as np
import pytest
import torch

from oracle import scan as orc

LN2 = np.log(2.0)


def test_scan_worked_example():
    # decay 1/2 a token; beta 1, 2, 1
    x, g = np.array([[[4.0], [3.0], [1.0]]]), np.full((1, 3, 1), -LN2)
    y, fin, _, _ = orc.scan(x, g, np.array([[[1.0], [2.0], [1.0]]]), np.array([[8.0]]))
    np.testing.assert_allclose(y[0, :, 0], [8, 10, 6], rtol=1e-15)
    assert fin[0, 0] == y[0, 2, 0]
    # a gate of minus infinity forgets everything; packed sequences do not mix, an empty one keeps its state
    y, fin, _, _ = orc.scan(x, np.array([[[-LN2], [-np.inf], [-LN2]]]), None, np.array([[8.0], [5.0], [2.0]]), [0, 2, 2, 3])
    np.testing.assert_allclose(y[0, :, 0], [8, 3, 2], rtol=1e-15)
    np.testing.assert_allclose(fin[:, 0], [3, 5, 2], rtol=1e-15)


def test_scan_is_linear_and_sums_decayed_inputs():
    r = np.random.default_rng(1)
    x, g, b = r.normal(size=(2, 6, 3)), -r.random((2, 6, 3)), r.random((2, 6, 3))
    y, _, _, _ = orc.scan(x, g, b)
    for t in range(6):
        want = sum(np.exp(g[:, j + 1:t + 1].sum(1)) * b[:, j] * x[:, j] for j in range(t + 1))
        np.testing.assert_allclose(y[:, t], want, rtol=1e-12)


def test_scan_steps_slots():
    x, g = np.array([[[1.0], [2.0], [3.0], [4.0]]]), np.full((1, 4, 1), -LN2)
    pool = np.array([[10.0], [20.0], [30.0], [40.0]])
    # the step before kept two tokens: starts from slot 2; column c takes the state after token c + 1, the last the last's
    y, after, _, _ = orc.scan_steps(x, g, pool, np.array([[0, 2, 3]]), num_accepted=[2])
    np.testing.assert_allclose(y[0, :, 0], [16, 10, 8, 8])
    np.testing.assert_allclose(after[:, 0], [16, 20, 10, 8])
    y, after, _, _ = orc.scan_steps(x, g, pool, np.array([[-1, 2, 3]]))
    assert not y.any() and (after == pool).all()


def test_scan_bwd_against_differences():
    r = np.random.default_rng(2)
    cu, D = [0, 4, 5, 5, 9], 3
    x, g, b = r.normal(size=(1, 9, D)), -r.random((1, 9, D)), r.random((1, 9, D))
    h0, dy, dht = r.normal(size=(4, D)), r.normal(size=(1, 9, D)), r.normal(size=(4, D))

    def loss(x, g, b, h0):
        y, fin, _, _ = orc.scan(x, g, b, h0, cu)
        return (y * dy).sum() + (fin * dht).sum()

    got = orc.scan_bwd(x, g, orc.scan(x, g, b, h0, cu)[0], dy, b, dht, h0, cu)
    for k, name in enumerate(("dx", "dg", "dbeta", "dinitial")):
        args, num = [x, g, b, h0], np.zeros_like((x, g, b, h0)[k])
        for i in np.ndindex(num.shape):
            e = np.zeros_like(num)
            e[i] = 1e-6
            hi, lo = ([a + s * e if j == k else a for j, a in enumerate(args)] for s in (1, -1))
            num[i] = (loss(*hi) - loss(*lo)) / 2e-6
        np.testing.assert_allclose(got[name][0], num, rtol=1e-6, atol=1e-8)
    assert "dbeta" not in orc.scan_bwd(None, g, dy, dy)


@pytest.mark.parametrize("bits,top", [(8, 127), (4, 7)])
def test_hold_promises(bits, top):
    r = np.random.default_rng(3)
    v = r.normal(size=(50, 100)) * np.exp(r.normal(size=(50, 1)) * 20)
    codes, scales = orc.hold(v, bits)
    assert codes.shape == v.shape and scales.shape == (50, 4) and np.abs(codes).max() == top
    s = np.repeat(scales, 32, -1)[:, :100]
    assert (np.abs(codes * s - v) <= s / 2).all()
    # scales are bf16 numbers, and the next one below does not reach
    b = torch.from_numpy(scales).to(torch.bfloat16)
    assert (b.double().numpy() == scales).all()
    below = (b.view(torch.int16) - 1).view(torch.bfloat16).double().numpy()
    high = np.stack([np.abs(v[:, k * 32:k * 32 + 32]).max(-1) for k in range(4)], -1)
    assert (top * scales >= high).all() and (top * below < high).all()


def test_hold_ties_zeros_and_not_finite():
    # largest 127: scale 1; halves go to the even side
    codes, scales = orc.hold(np.array([[127.0, 0.5, 1.5, -2.5, 2.5000001, -0.5000001, 63.5]]))
    assert scales.tolist() == [[1.0]] and codes.tolist() == [[127, 0, 2, -2, 3, -1, 64]]
    codes, scales = orc.hold(np.array([[127.1] + [0.0] * 31 + [1e-31, -2e-31]]))
    assert scales.tolist() == [[1.0078125, 0.0]] and codes[0, 32:].tolist() == [0, 0]
    for bad in (np.inf, -np.inf, np.nan):
        codes, scales = orc.hold(np.array([[1.0] * 32 + [bad, 2.0]]))
        assert scales[0, 0] > 0 and np.isnan(scales[0, 1]) and not codes[0, 32:].any()
        assert np.isnan(orc.restore(codes, scales)[0, 32:]).all()
    assert orc.pack4(np.array([[1, -1, 7, -7, 3]])).tolist() == [[0xf1, 0x97, 0x03]]
