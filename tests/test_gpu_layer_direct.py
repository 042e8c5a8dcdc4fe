"""The direct calls of the C entry points (status codes, the caller's own structs,
outputs, workspace and stream) against the functions of the package, bit for bit.
"""
import pytest
import torch

from test_gpu_layer import BF, DEV, F32, Draw, _conv_inputs, _gdn, _steps_inputs

pytestmark = pytest.mark.gpu


def _parts(tensors):
    from gated_deltanet_chunked_delta_amd import gdn_conv_pieces
    p = gdn_conv_pieces()
    for i, t in enumerate(tensors):
        p.ptr[i], p.dim[i] = t.data_ptr(), t.shape[-1]
    return p


def _code(dtype):
    return {BF: 0, F32: 1}[dtype]


def _same(*pairs):
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in pairs)


@pytest.mark.parametrize("own_stream", [False, True])
def test_direct_calls_of_the_steps(own_stream):
    gdn = _gdn()
    x = {k: None if t is None else t.to(DEV) for k, t in _steps_inputs("verify", BF).items()}
    pools = [x["pool"].clone(), x["pool"].clone()]
    want = gdn.fused_recurrent_gated_delta_rule_steps(x["q"], x["k"], x["v"], None, None, pools[0], x["idx"], num_accepted=x["acc"],
                                                      use_qk_l2norm_in_kernel=True, A_log=x["A_log"], dt_bias=x["dt_bias"],
                                                      a_raw=x["a"], b_raw=x["b"])
    out = torch.empty_like(x["v"])
    B, T, H, K = x["q"].shape
    shape = gdn.make_shape(B=B, T=T, H=H, HV=x["v"].shape[2], K=K, V=x["v"].shape[3], N=B, dtype=_code(BF))
    gates = gdn.make_gates(x["A_log"], x["dt_bias"], x["a"], x["b"])
    torch.cuda.synchronize()
    stream = torch.cuda.Stream().cuda_stream if own_stream else None
    pool = gdn.make_step_pool(pools[1], x["idx"], x["acc"])
    st = gdn.gdn_recurrent_steps(x["q"], x["k"], x["v"], None, None, gates, K ** -0.5, True, pool, None, out, shape, stream)
    assert st == gdn.GDN_OK
    _same((out, want), (pools[1], pools[0]))
    assert gdn.gdn_recurrent_steps(x["q"], x["k"], x["v"], None, None, gates, 1.0, True, pool, None, None, shape) == -1
    one = gdn.make_step_pool(pools[1], x["idx"][:, 0].contiguous())
    assert one.cols == 1 and one.num_accepted is None and one.pool_size == pools[1].shape[0] and one.dtype == _code(pools[1].dtype)


@pytest.mark.parametrize("own_stream", [False, True])
def test_direct_calls_of_the_convolution(own_stream):
    gdn = _gdn()
    x = _conv_inputs("packed", BF)
    xs, w, b, h0, cu, split = (x[n] for n in ("x", "w", "b", "h0", "cu", "split"))
    N, D, W1 = h0.shape
    T = xs.shape[1]
    shape = gdn.gdn_conv_shape(1, T, D, W1 + 1, N, 0, 0, xs.stride(1))
    new = lambda: [torch.empty(1, T, n, dtype=BF, device=DEV) for n in split]
    d = x["draw"]
    idx = d.slots(N + 2, N).to(DEV)
    pool0 = d.randn(N + 2, D, W1, dtype=BF).to(DEV)
    dys = [t.contiguous() for t in x["dy"].split(split, -1)]
    want, final = gdn.causal_conv1d(xs, w, b, initial_state=h0, cu_seqlens=cu, split_sizes=split)
    pools = [pool0.clone() for _ in range(4)]
    want_pool, _ = gdn.causal_conv1d(xs, w, b, cu_seqlens=cu, split_sizes=split, conv_state_pool=pools[0], conv_state_indices=idx)
    want_step = gdn.causal_conv1d_update(xs, w, pools[2], idx, b, cu_seqlens=cu, split_sizes=split)
    grads = gdn.causal_conv1d_bwd(xs, w, dys, b, initial_state=h0, cu_seqlens=cu, output_dinitial=True)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream().cuda_stream if own_stream else None
    outs, fin = [new() for _ in range(3)], torch.empty_like(h0)
    assert gdn.gdn_conv_fwd(xs, w, b, True, h0, cu, _parts(outs[0]), fin, shape, stream) == 0
    _same((fin, final), *zip(outs[0], want))
    assert gdn.gdn_conv_fwd_pool(xs, w, b, True, gdn.make_state_pool(pools[1], idx, True), cu, _parts(outs[1]), shape, stream) == 0
    _same((pools[1], pools[0]), *zip(outs[1], want_pool))
    assert gdn.gdn_conv_update(xs, w, b, True, gdn.make_step_pool(pools[3], idx), cu, _parts(outs[2]), shape, stream) == 0
    _same((pools[3], pools[2]), *zip(outs[2], want_step))
    got = [torch.empty_like(g) for g in grads]
    ws = torch.empty(gdn.gdn_conv_bwd_workspace_bytes(shape), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert gdn.gdn_conv_bwd(xs, w, b, True, h0, cu, _parts(dys), *got, shape, ws, stream=stream) == 0
    _same(*zip(got, grads))
    assert gdn.gdn_conv_bwd(xs, w, b, True, h0, cu, _parts(dys), *got, shape, ws, workspace_bytes=16) == -5
    assert gdn.gdn_conv_bwd(xs, w, b, True, h0, cu, _parts(dys), *got, shape, None) == -5
    assert gdn.gdn_conv_fwd(None, w, b, True, h0, cu, _parts(outs[0]), fin, shape, 0) == -1


@pytest.mark.parametrize("own_stream", [False, True])
def test_direct_calls_of_the_norms(own_stream):
    gdn = _gdn()
    d = Draw(4)
    rows, D = 70, 250
    x, z, res, dy, dh = (d.randn(rows, D, dtype=BF).to(DEV) for _ in range(5))
    w = d.randn(D, dtype=BF).to(DEV)
    shape = gdn.gdn_norm_shape(rows, D, D, 1, 0, 0)
    y = gdn.fused_gated_rms_norm(x, z, w)
    gated = gdn.fused_gated_rms_norm_bwd(x, z, w, dy)
    y2, hidden = gdn.fused_add_rms_norm(x, res, w, residual_scale=0.5, weight_offset=1.0)
    add = gdn.fused_add_rms_norm_bwd(dy, dh, hidden, w, residual_scale=0.5, weight_offset=1.0)
    outs = [torch.empty_like(x) for _ in range(7)]
    dws = [torch.empty(D, device=DEV) for _ in range(2)]
    ws = torch.empty(gdn.gdn_norm_bwd_workspace_bytes(shape), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream().cuda_stream if own_stream else None
    assert gdn.gdn_gated_norm(x, z, w, 1e-6, outs[0], shape, stream) == 0
    assert gdn.gdn_gated_norm_bwd(x, z, w, 1e-6, dy, outs[1], outs[2], dws[0], shape, ws, stream=stream) == 0
    assert gdn.gdn_add_norm(x, res, w, 0.5, 1.0, 1e-6, outs[3], outs[4], shape, stream) == 0
    assert gdn.gdn_add_norm_bwd(dy, dh, hidden, w, 0.5, 1.0, 1e-6, outs[5], outs[6], dws[1], shape, ws, stream=stream) == 0
    _same((outs[0], y), (outs[1], gated[0]), (outs[2], gated[1]), (dws[0], gated[2]), (outs[3], y2), (outs[4], hidden),
          (outs[5], add[0]), (outs[6], add[1]), (dws[1], add[2]))
    assert gdn.gdn_gated_norm(x, z, w, 1e-6, None, shape) == -1
    assert gdn.gdn_gated_norm_bwd(x, z, w, 1e-6, dy, outs[1], outs[2], dws[0], shape, ws, workspace_bytes=8) == -5
    assert gdn.gdn_add_norm(x, res, w, 0.5, 1.0, 1e-6, None, None, shape) == -1
    assert gdn.gdn_add_norm_bwd(dy, dh, hidden, w, 0.5, 1.0, 1e-6, None, None, dws[1], shape, ws) == -1
