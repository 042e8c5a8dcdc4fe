"""Pins of the float64 definitions in oracle/layer.py (no GPU): worked examples,
the recurrence oracle, and central differences of the forward functions."""
import numpy as np
import pytest
import torch

import oracle
from oracle import layer


def test_conv_worked_example():
    # width 3, one column, weights 1, 10, 100 on x[t-2], x[t-1], x[t]; no SiLU
    x = np.array([[[1.0], [2.0], [3.0], [4.0]]])
    w = np.array([[1.0, 10.0, 100.0]])
    y, final, _ = layer.conv(x, w, silu=False)
    assert y[0, :, 0].tolist() == [100, 210, 321, 432] and final[0, 0].tolist() == [3, 4]
    # a history 5, 6 in front (5 the older), a bias, and SiLU
    y, _, _ = layer.conv(x, w, np.array([0.5]), np.array([[[5.0, 6.0]]]), silu=False)
    assert y[0, :2, 0].tolist() == [5 + 60 + 100 + 0.5, 6 + 10 + 200 + 0.5]
    y, _, _ = layer.conv(np.array([[[0.01]]]), w)
    assert abs(y[0, 0, 0] - 1 / (1 + np.exp(-1.0))) < 1e-15
    # two packed sequences and an empty one: no mixing over the border
    y, final, _ = layer.conv(x, w, cu_seqlens=[0, 2, 2, 4], silu=False)
    assert y[0, :, 0].tolist() == [100, 210, 300, 430]
    assert final[:, 0].tolist() == [[1, 2], [0, 0], [3, 4]]


def test_conv_update_slots():
    x = np.arange(1.0, 5.0).reshape(1, 4, 1)
    w = np.array([[1.0, 10.0, 100.0]])
    pool = np.array([[[7.0, 8.0]], [[0.0, 0.0]], [[5.0, 6.0]], [[9.0, 9.0]]])
    # three columns, the step before kept two tokens: starts from slot 2; the last column takes the last token's
    y, after, _ = layer.conv_update(x, w, pool, np.array([[0, 2, 3]]), num_accepted=[2], silu=False)
    assert y[0, :, 0].tolist() == [5 + 60 + 100, 6 + 10 + 200, 321, 432]
    assert after[:, 0].tolist() == [[6, 1], [0, 0], [1, 2], [3, 4]]
    # padding: zeros, nothing stored; a slot to write outside the pool is skipped
    y, after, _ = layer.conv_update(x, w, pool, np.array([[-1, 2, 3]]), silu=False)
    assert not y.any() and (after == pool).all()
    y, after, _ = layer.conv_update(x, w, pool, np.array([[0, 4, 3]]), silu=False)
    assert after[:, 0].tolist() == [[8, 1], [0, 0], [5, 6], [3, 4]]
    # fewer tokens than columns: the columns behind stay
    _, after, _ = layer.conv_update(x[:, :1], w, pool, np.array([[0, 2, 3]]), silu=False)
    assert after[:, 0].tolist() == [[8, 1], [0, 0], [5, 6], [9, 9]]


def test_norm_worked_examples():
    y, _ = layer.gated_norm(np.array([[3.0, 4.0]]), np.array([[0.0, np.log(3.0)]]), np.array([1.0, 2.0]), eps=0.0)
    # rms = sqrt(12.5); silu(0) = 0, silu(ln 3) = 0.75 ln 3
    np.testing.assert_allclose(y, [[0.0, 4 / np.sqrt(12.5) * 2 * 0.75 * np.log(3.0)]], rtol=1e-15)
    y, h = layer.add_norm(np.array([[2.0, 4.0]]), np.array([[2.0, 2.0]]), np.array([0.0, 1.0]), eps=0.0,
                          residual_scale=0.5, weight_offset=1.0)
    assert h.tolist() == [[3.0, 4.0]]
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)


@pytest.mark.parametrize("l2", [True, False])
def test_steps_match_the_recurrence_oracle(l2):
    r = np.random.default_rng(3)
    H, HV, K, V, N, T = 2, 4, 64, 64, 3, 5
    q, k = (r.normal(size=(N, T, H, K)).astype(np.float32) * (1 if l2 else K ** -0.5) for _ in range(2))
    v, g = r.normal(size=(N, T, HV, V)).astype(np.float32), -r.random((N, T, HV)).astype(np.float32)
    beta = r.random((N, T, HV)).astype(np.float32)
    pool = r.normal(size=(8, HV, K, V)).astype(np.float32)
    idx = np.array([4, 7, 1])
    o, fin = oracle.recurrent(q, k, v, g, beta, initial_state=pool[idx], use_l2norm=l2)
    out, after, _ = layer.steps(q, k, v, g, beta, pool, idx, use_l2norm=l2)
    np.testing.assert_allclose(out, o, atol=1e-12)
    np.testing.assert_allclose(after[idx], fin, atol=1e-12)
    rest = [i for i in range(8) if i not in idx]
    assert (after[rest] == pool[rest]).all()
    # every column: the state after each prefix
    cols = np.array([[4, 0, 2], [7, 3, 5], [1, 6, -1]])
    out, after, _ = layer.steps(q, k, v, g, beta, pool, cols, use_l2norm=l2)
    np.testing.assert_allclose(out, o, atol=1e-12)
    for c, upto in ((0, 1), (1, 2), (2, T)):
        _, fin = oracle.recurrent(q[:, :upto], k[:, :upto], v[:, :upto], g[:, :upto], beta[:, :upto],
                                  initial_state=pool[idx], use_l2norm=l2)
        for n in range(N):
            if cols[n, c] >= 0:
                np.testing.assert_allclose(after[cols[n, c]], fin[n], atol=1e-12)
    # an accepted count outside [1, cols] is taken into it
    a = layer.steps(q, k, v, g, beta, pool, cols, num_accepted=[0, 9, 2], use_l2norm=l2)[0]
    b = layer.steps(q, k, v, g, beta, pool, cols, num_accepted=[1, 3, 2], use_l2norm=l2)[0]
    assert (a == b).all()


def _differences(f, args, at, cot, h=1e-6):
    """Central differences of sum(cot * f(args)) by args[at]."""
    x = args[at]
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        y = []
        for s in (h, -h):
            z = x.copy()
            z[i] += s
            y.append(sum((c * o).sum() for c, o in zip(cot, f(*args[:at], z, *args[at + 1:]))))
        g[i] = (y[0] - y[1]) / (2 * h)
    return g


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_gradients_by_differences(W, silu):
    r = np.random.default_rng(W)
    D, cu = 3, [0, 1, 1, 6, 8]
    x, w, b = r.normal(size=(1, 8, D)), r.normal(size=(D, W)), r.normal(size=D)
    init, dy = r.normal(size=(4, D, W - 1)), r.normal(size=(1, 8, D))
    f = lambda x, w, b, i: layer.conv(x, w, b, i, cu, silu)[:1]
    got = layer.conv_bwd(x, w, dy, b, init, cu, silu)
    for at, name in enumerate(("dx", "dweight", "dbias", "dinitial")):
        np.testing.assert_allclose(got[name][0], _differences(f, [x, w, b, init], at, [dy]), atol=1e-7)
        assert (got[name][1] >= np.abs(got[name][0]) - 1e-12).all()


def test_norm_gradients_by_differences():
    r = np.random.default_rng(7)
    x, z, w, dy = r.normal(size=(2, 3, 5)), r.normal(size=(2, 3, 5)), r.normal(size=5), r.normal(size=(2, 3, 5))
    f = lambda x, z, w: layer.gated_norm(x, z, w)[:1]
    got = layer.gated_norm_bwd(x, z, w, dy)
    for at, name in enumerate(("dx", "dz", "dweight")):
        np.testing.assert_allclose(got[name][0], _differences(f, [x, z, w], at, [dy]), atol=1e-7)
    dh = r.normal(size=(2, 3, 5))
    f = lambda x, res, w: layer.add_norm(x, res, w, residual_scale=0.3, weight_offset=1.0)
    got = layer.add_norm_bwd(dy, dh, f(x, z, w)[1], w, residual_scale=0.3, weight_offset=1.0)
    for at, name in enumerate(("dx", "dresidual", "dweight")):
        np.testing.assert_allclose(got[name][0], _differences(f, [x, z, w], at, [dy, dh]), atol=1e-7)


def test_definitions_agree_with_torch_autograd():
    torch.manual_seed(1)
    x, w, b = torch.randn(2, 7, 5, dtype=torch.float64), torch.randn(5, 4, dtype=torch.float64), torch.randn(5, dtype=torch.float64)
    y = torch.nn.functional.silu(torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (3, 0)),
                                                            w[:, None], b, groups=5)).transpose(1, 2)
    np.testing.assert_allclose(layer.conv(x, w, b)[0], y.numpy(), atol=1e-13)
