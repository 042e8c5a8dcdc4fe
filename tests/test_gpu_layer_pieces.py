"""A decode layer operator by operator, each fed what the run gave it, against the
float64 definitions.

Bars as for the single operators: fp32 arithmetic, each output rounded once.  For
the steps a state is off by at most 64 2^-24 of the oracle's bound (which is at
least its norm); an output, its inner product with a unit q times the scale, has
24 roundings of its own and the product's three: 64 + 27 < 128.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import layer
from test_gpu_layer import BF, DEV, F32, ULP, Draw, _gdn, _layer, _near, _np, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_decode_layer_piece_by_piece(dtype):
    gdn = _gdn()
    N, T, cols = 6, 3, 3
    (H, HV, K, V, D), t = _layer(1, N, T, dtype)
    P, d = N * cols + 2, Draw(9)
    idx = d.slots(P, N * cols).view(N, cols)
    idx[4] = -1
    acc = torch.tensor([1, 2, 3, 1, 2, 3], dtype=torch.int32)
    conv0, state0 = d.randn(P, D, 3, dtype=dtype), d.randn(P, HV, K, V, std=0.1)
    conv, state, res = conv0.to(DEV), state0.to(DEV), t["res"].clone()
    slots, kept = idx.to(DEV), acc.to(DEV)
    _say(f"[layer] decode piece by piece {dtype}")

    y, hidden = gdn.fused_add_rms_norm(t["x"], res, t["w_in"], weight_offset=1.0, hidden=res)
    ref, h = layer.add_norm(t["x"], t["res"], t["w_in"], weight_offset=1.0)
    size = np.abs(_np(t["x"])) + np.abs(_np(t["res"]))
    _near("hidden", hidden, h, size, 2)
    _near("y", y, ref, np.abs(ref) + size * np.abs(_np(t["w_in"]) + 1) / np.sqrt((h * h).mean(-1, keepdims=True) + 1e-6), 64)

    p = (y.float().view(N * T, -1) @ t["proj"].float()).to(dtype).view(N, T, -1)
    qkv, z, a, b = p.split((D, HV * V, HV, HV), -1)
    parts = gdn.causal_conv1d_update(qkv, t["conv"], conv, slots, num_accepted=kept, split_sizes=(H * K, H * K, HV * V))
    ref, after, mag = layer.conv_update(qkv, t["conv"], conv0, idx, num_accepted=acc)
    _near("q, k, v", torch.cat(parts, -1), ref, mag, 8)
    assert (_np(conv) == after).all()

    q, k, v = parts[0].view(N, T, H, K), parts[1].view(N, T, H, K), parts[2].view(N, T, HV, V)
    a, b = a.contiguous(), b.contiguous()
    o = gdn.fused_recurrent_gated_delta_rule_steps(q, k, v, None, None, state, slots, num_accepted=kept, use_qk_l2norm_in_kernel=True,
                                                   A_log=t["A_log"], dt_bias=t["dt_bias"], a_raw=a, b_raw=b)
    g, beta = oracle.gating(t["A_log"].cpu(), t["dt_bias"].cpu(), a.cpu(), b.cpu())
    ref, after, bound = layer.steps(q, k, v, g, beta, state0, idx, acc, use_l2norm=True)
    err, size = np.linalg.norm(_np(o) - ref, axis=-1), np.linalg.norm(ref, axis=-1)
    assert (err <= K ** -0.5 * 128 * ULP * bound[:, None] + torch.finfo(dtype).eps / 2 * 1.01 * size + 1e-30).all()
    err = np.sqrt(((_np(state) - after) ** 2).sum((-2, -1)))
    assert (err <= 64 * ULP * bound.max(0)).all()
    untouched = [s for s in range(P) if s not in idx.flatten().tolist()]
    assert untouched and (_np(state)[untouched] == _np(state0)[untouched]).all()
    assert not o[4].any() and not any(u[4].any() for u in parts)

    zs = z.unflatten(-1, (HV, V))
    _near("out", gdn.fused_gated_rms_norm(o, zs, t["w_out"].to(dtype)), *layer.gated_norm(o, zs, t["w_out"].to(dtype)), 64)


def test_prompts_on_the_pool_in_a_graph():
    """A packed prefill of the convolution on its pool, captured: the final states' launch overwrites the histories
    that the strips read, on every replay; sequences over many strips, padding rows and an empty sequence."""
    gdn = _gdn()
    d, lens, D = Draw(17), [1, 700, 0, 3, 1290, 2, 64], 1040
    N, T = len(lens), sum(lens)
    x, w = d.randn(1, T, D, dtype=BF).to(DEV), d.randn(D, 4, std=0.5, dtype=BF).to(DEV)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV)
    idx = torch.tensor([3, 0, 7, -1, 5, 9, 2], dtype=torch.int32, device=DEV)     # 9 lies outside
    pool0 = d.randn(8, D, 3, dtype=BF).to(DEV)
    pool = pool0.clone()
    step = lambda: gdn.causal_conv1d(x, w, cu_seqlens=cu, conv_state_pool=pool, conv_state_indices=idx)[0]
    runs = []
    for _ in range(2):     # from pool0, then from what the first run left
        y = step()
        runs.append((y.clone(), pool.clone()))
    start = torch.stack([pool0[i] if 0 <= i < 8 else torch.zeros_like(pool0[0]) for i in idx.tolist()])
    want, final = gdn.causal_conv1d(x, w, initial_state=start, cu_seqlens=cu)
    assert torch.equal(runs[0][0], want) and torch.equal(runs[0][1][idx[idx.ge(0) & idx.lt(8)].long()],
                                                         final[idx.ge(0) & idx.lt(8)])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        pool.copy_(pool0)
        for want in runs:
            out.fill_(7)
            torch.randn(1 << 20, device=DEV).mul_(2.0).sum().item()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(pool, want[1]), f"replay {i}"
