"""The linear recurrence, state caches and checkpoints as they are used together, and
at the edges: padded batches, values that are not finite, offsets beyond 32 bits,
captured graphs, other streams, slots named twice."""
import numpy as np
import pytest
import torch

from oracle import layer
from oracle import scan as orc

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ULP = 2.0 ** -24


def _gdn():
    import gated_deltanet_chunked_delta_amd as gdn
    gdn.load_library()
    return gdn


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(name, got, ref, mag, c):
    half = torch.finfo(got.dtype).eps / 2
    tol = c * ULP * mag + half * (np.abs(ref) + c * ULP * mag) + 1e-36
    over = np.abs(_np(got) - ref) / tol
    print(f"    {name}: worst error {float(over.max()):.2f} of the bar", flush=True)
    assert np.isfinite(over).all() and over.max() <= 1.0, name


class Draw:
    def __init__(self, seed):
        self.gen = torch.Generator().manual_seed(seed)

    def randn(self, *shape, std=1.0, dtype=F32):
        return (torch.randn(*shape, generator=self.gen) * std).to(dtype).to(DEV)

    def gates(self, *shape, dtype=F32):
        return (-torch.nn.functional.softplus(torch.randn(*shape, generator=self.gen)) * 0.2).to(dtype).to(DEV)

    def rand(self, *shape, dtype=F32):
        return torch.rand(*shape, generator=self.gen).to(dtype).to(DEV)


def _cu(*lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=I32, device=DEV)


def test_a_layer_of_the_recurrence():
    """Convolution, gates, recurrence on a pool, norm that keeps its inputs; the gradients back through them, the
    recurrence's from the norm's checkpoint; the states into a cache of 8 bits, back into other slots, and on token by token."""
    gdn = _gdn()
    d = Draw(3)
    heads, dim, lens = 6, 64, (90, 1, 300)
    D, T, N = heads * dim, sum(lens), len(lens)
    cu = _cu(*lens)
    xin, w = d.randn(1, T, D, dtype=BF), d.randn(D, 4, std=0.5, dtype=BF)
    A_log, dt_bias, a, b = d.rand(D) - 2, d.rand(D), d.randn(1, T, D, dtype=BF), d.randn(1, T, D, dtype=BF)
    z, wn = d.randn(1, T, heads, dim, dtype=BF), (d.randn(dim, std=0.2) + 1).to(BF)
    x, _ = gdn.causal_conv1d(xin, w, cu_seqlens=cu)
    g, beta = gdn.fused_gdn_gating(A_log, a, b, dt_bias)
    g, beta = g.view(1, T, D), beta.view(1, T, D)
    pool, slots = torch.zeros(5, D, device=DEV), torch.tensor([3, 0, 4], dtype=I32, device=DEV)
    y, _ = gdn.gated_linear_recurrence(x, g, beta, cu_seqlens=cu, state_pool=pool, state_indices=slots,
                                       read_initial_state=False)
    ref, fin, mag, mfin = orc.scan(x, g, beta, None, cu)
    _near("y", y, ref, mag, 5)
    _near("states", pool[slots.long()], fin, mfin, 5)
    out, y8, z8 = gdn.fused_gated_rms_norm_checkpoint(y.view(1, T, heads, dim), z, wn)
    nref, nmag = layer.gated_norm(y.view(1, T, heads, dim), z, wn)
    _near("out", out, nref, nmag, 64)
    # backward: the norm's x checkpoint is the recurrence's y checkpoint
    dout = d.randn(1, T, heads, dim, dtype=BF)
    dy, dz, dwn = gdn.fused_gated_rms_norm_checkpoint_bwd(y8, z8, wn, dout)
    yr, zr = (torch.from_numpy(orc.restore(*c)) for c in (y8, z8))
    for t, n, c in zip((dy, dz, dwn), ("dx", "dz", "dweight"), (128, 128, 256)):
        _near("norm " + n, t, *layer.gated_norm_bwd(yr, zr, wn, dout)[n], c)
    x8 = gdn.checkpoint_activation(x)
    got = gdn.gated_linear_recurrence_bwd(x8, g, y8, dy.view(1, T, D), beta, cu_seqlens=cu)
    grads = orc.scan_bwd(torch.from_numpy(orc.restore(*x8)), g, yr.view(1, T, D), dy.view(1, T, D), beta, None, None, cu)
    for t, n in zip(got, ("dx", "dg", "dbeta")):
        _near(n, t, *grads[n], 8)
    again = gdn.gated_linear_recurrence_bwd(x8, g, gdn.checkpoint_activation(y), dy.view(1, T, D), beta, cu_seqlens=cu)
    assert all(u is v is None or torch.equal(u, v) for u, v in zip(got, again))
    da, db, dA, ddt = gdn.fused_gdn_gating_bwd(A_log, a, b, dt_bias, got[1].view(a.shape), got[2].view(a.shape))
    assert all(t.isfinite().all() for t in (da, db, dA, ddt))
    # the requests leave and come back to other slots, their states within half a step of what they were
    codes, scales = gdn.make_state_cache(pool, 4)
    at, back = torch.tensor([2, 0, 3], dtype=I32, device=DEV), torch.tensor([1, 2, 0], dtype=I32, device=DEV)
    gdn.state_cache_write(pool, slots, codes, scales, at)
    later = torch.full_like(pool, 7.0)
    gdn.state_cache_read(codes, scales, at, later, back)
    held = orc.restore(*orc.hold(pool[slots.long()]))
    assert (_np(later[back.long()]) == held).all() and (later[3:] == 7.0).all()
    step = d.randn(N, 2, D, dtype=BF), d.gates(N, 2, D), d.rand(N, 2, D)
    y2 = gdn.gated_linear_recurrence_steps(step[0], step[1], later, back, beta=step[2])
    ref2, fin2, mag2, mfin2 = orc.scan(*step, torch.from_numpy(held))
    _near("steps", y2, ref2, mag2, 5)
    _near("stepped states", later[back.long()], fin2, mfin2, 5)


def test_delta_rule_states_through_a_cache():
    """A prefix's delta-rule states, held in 8 bits, start a prefill from a pool as the values they stand for do."""
    gdn = _gdn()
    d = Draw(4)
    H, HV, K, V, T = 1, 2, 64, 128, 70
    q, k = d.randn(1, T, H, K, dtype=BF), d.randn(1, T, H, K, dtype=BF)
    v, g, beta = d.randn(1, T, HV, V, dtype=BF), d.gates(1, T, HV), d.rand(1, T, HV)
    pool, one = torch.zeros(3, HV, K, V, device=DEV), torch.tensor([1], dtype=I32, device=DEV)
    gdn.chunk_gated_delta_rule(q, k, v, g, beta, use_qk_l2norm_in_kernel=True, ssm_state_pool=pool, ssm_state_indices=one)
    for bits, part in ((8, 1 / 120), (4, 1 / 6.9)):
        codes, scales = gdn.make_state_cache(pool, 2, bits)
        gdn.state_cache_write(pool, one, codes, scales, one * 0)
        back = torch.zeros_like(pool)
        gdn.state_cache_read(codes, scales, one * 0, back, one + 1)
        rows = pool[1].view(-1, 32)
        assert ((back[2].view(-1, 32) - rows).abs() <= rows.abs().amax(1, keepdim=True) * part / 2).all()
        start = back[2:].clone()
        o1, _ = gdn.chunk_gated_delta_rule(q, k, v, g, beta, use_qk_l2norm_in_kernel=True, ssm_state_pool=back,
                                            ssm_state_indices=one + 1)
        o2, f2 = gdn.chunk_gated_delta_rule(q, k, v, g, beta, use_qk_l2norm_in_kernel=True, initial_state=start)
        assert torch.equal(o1, o2) and torch.equal(back[2:], f2)


@pytest.mark.parametrize("dtype,gate", [(BF, F32), (BF, BF), (F32, F32)], ids=["bf16_fp32", "bf16", "fp32"])
def test_rows_behind_the_last_sequence(dtype, gate):
    """A batch padded to a fixed T: the rows behind the last sequence, NaN here, are not read, and what their outputs
    held stays; the others are the bits of the batch without them."""
    gdn = _gdn()
    d = Draw(5)
    lens, D, T = (130, 0, 77), 70, 700
    cu, used = _cu(*lens), sum(lens)
    nan = float("nan")
    x, g, b = d.randn(1, T, D, dtype=dtype), d.gates(1, T, D, dtype=gate), d.rand(1, T, D, dtype=gate)
    for t in (x, g, b):
        t[:, used:] = nan
    h0 = d.randn(3, D)
    cut = [t[:, :used].contiguous() for t in (x, g, b)]
    out = torch.full_like(x, 9.0)
    y, f = gdn.gated_linear_recurrence(x, g, b, initial_state=h0, cu_seqlens=cu, out=out)
    y1, f1 = gdn.gated_linear_recurrence(*cut, initial_state=h0, cu_seqlens=cu)
    assert torch.equal(y[:, :used], y1) and torch.equal(f, f1) and (y[:, used:] == 9.0).all() and torch.equal(f1[1], h0[1])
    dy = d.randn(1, T, D, dtype=dtype)
    dy[:, used:] = nan
    ypad = y.clone()
    ypad[:, used:] = nan
    a = gdn.gated_linear_recurrence_bwd(x, g, ypad, dy, b, initial_state=h0, cu_seqlens=cu, output_dinitial=True)
    e = gdn.gated_linear_recurrence_bwd(cut[0], cut[1], y1, dy[:, :used].contiguous(), cut[2], initial_state=h0, cu_seqlens=cu,
                                        output_dinitial=True)
    for s, t in zip(a[:3], e[:3]):
        assert torch.equal(s[:, :used], t)
    assert torch.equal(a[3], e[3])
    pool = d.randn(4, D)
    idx = torch.tensor([2, 0, 3], dtype=I32, device=DEV)
    p1, p2 = pool.clone(), pool.clone()
    out.fill_(9.0)
    s1 = gdn.gated_linear_recurrence_steps(x, g, p1, idx, beta=b, cu_seqlens=cu, out=out)
    s2 = gdn.gated_linear_recurrence_steps(cut[0], cut[1], p2, idx, beta=cut[2], cu_seqlens=cu)
    assert torch.equal(s1[:, :used], s2) and (s1[:, used:] == 9.0).all() and torch.equal(p1, p2)


@pytest.mark.parametrize("gate", [F32, BF], ids=["fp32", "bf16"])
def test_what_is_not_finite_stays_in_its_sequence(gate):
    """Infinities and NaNs of one sequence do not reach another, in whatever tile; gates of the lowest value and of
    minus infinity forget everything that is finite."""
    gdn = _gdn()
    d = Draw(6)
    lens, D = (3, 200, 5, 1, 700, 64, 9), 37
    cu, T, N = _cu(*lens), sum(lens), len(lens)
    x, g, b = d.randn(1, T, D, dtype=BF), d.gates(1, T, D, dtype=gate), d.rand(1, T, D, dtype=gate)
    h0, dht, dy = d.randn(N, D), d.randn(N, D), d.randn(1, T, D, dtype=BF)

    def both(x, g, h0, dy, dht):
        y, f = gdn.gated_linear_recurrence(x, g, b, initial_state=h0, cu_seqlens=cu)
        return (y, f, *gdn.gated_linear_recurrence_bwd(x, g, y, dy, b, dht=dht, initial_state=h0, cu_seqlens=cu, output_dinitial=True))

    clean = both(x, g, h0, dy, dht)
    starts = np.cumsum([0] + list(lens))
    for n in (1, 3, 4):
        for value in (float("nan"), float("inf")):
            bad = [t.clone() for t in (x, g, h0, dy, dht)]
            s = slice(starts[n], starts[n + 1])
            bad[0][:, s], bad[2][n], bad[3][:, s], bad[4][n] = value, value, value, value
            if value != value:
                bad[1][:, s] = value
            got = both(*bad)
            rows = torch.ones(T, dtype=torch.bool, device=DEV)
            rows[s] = False
            seqs = torch.arange(N, device=DEV) != n
            for i, (u, v) in enumerate(zip(got, clean)):
                u, v = (u[seqs], v[seqs]) if u.dim() == 2 else (u[:, rows], v[:, rows])
                assert torch.equal(u, v), (n, value, i)
            assert not got[0][:, s].isfinite().any() and not got[2][:, s].isfinite().any()
    for low in (-float("inf"), torch.finfo(gate).min):
        g2 = g.clone()
        g2[:, 300] = low                     # inside the long sequence
        y, f = gdn.gated_linear_recurrence(x, g2, b, initial_state=h0, cu_seqlens=cu)
        u = (x[:, 300].float() * b[:, 300].float()).to(BF)
        assert torch.equal(y[:, 300], u) and y.isfinite().all() and f.isfinite().all()
        grads = gdn.gated_linear_recurrence_bwd(x, g2, y, dy, b, dht=dht, initial_state=h0, cu_seqlens=cu)
        assert all(t.isfinite().all() for t in grads[:3]) and not grads[1][:, 300].any()


def test_rows_beyond_32_bits():
    """More than 2^31 elements: the rows behind a token that forgets everything are the bits of the call on them alone."""
    gdn = _gdn()
    T, D = 540_000, 4096
    tail = 700
    x = torch.randn(1, T, D, device=DEV, dtype=BF)
    g = torch.full((1, T, D), -0.05, device=DEV, dtype=BF)
    g[:, T - tail] = -float("inf")
    y, f = gdn.gated_linear_recurrence(x, g)
    part = slice(T - tail, T)
    y1, f1 = gdn.gated_linear_recurrence(x[:, part].contiguous(), g[:, part].contiguous())
    # the same sums, but in tiles that begin at other tokens
    torch.testing.assert_close(y[:, part], y1, rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(f, f1, rtol=0, atol=2e-5)
    del x
    dy = torch.zeros(1, T, D, device=DEV, dtype=BF)
    dy[:, part] = torch.randn(1, tail, D, device=DEV, dtype=BF)
    dx, dg, _, _ = gdn.gated_linear_recurrence_bwd(None, g, y, dy)
    ex, eg, _, _ = gdn.gated_linear_recurrence_bwd(None, g[:, part].contiguous(), y1, dy[:, part].contiguous())
    torch.testing.assert_close(dx[:, part], ex, rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(dg[:, part], eg, rtol=2.0 ** -6, atol=1e-4)
    assert not dx[:, :T - tail].any() and not dg[:, :T - tail].any()


def test_captured_graphs_that_share_a_workspace():
    """Two graphs, their calls given one workspace, replayed in turn with eager work between: each replay gives the
    bits of the eager calls on the inputs of that moment."""
    gdn = _gdn()
    d = Draw(8)
    T, D, N = 900, 200, 3
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)
    x, g, b, dy = d.randn(1, T, D, dtype=BF), d.gates(1, T, D), d.rand(1, T, D), d.randn(1, T, D, dtype=BF)
    cu, h0 = _cu(400, 0, 500), d.randn(N, D)
    pool, idx = d.randn(5, D), torch.tensor([4, 1, 2], dtype=I32, device=DEV)
    codes, scales = gdn.make_state_cache(pool, 5, 4)
    z, w = d.randn(1, T, 2, 100, dtype=BF), d.rand(100).to(BF)

    def first():
        y, f = gdn.gated_linear_recurrence(x, g, b, initial_state=h0, cu_seqlens=cu, workspace=ws)
        o, y8, z8 = gdn.fused_gated_rms_norm_checkpoint(y.view(1, T, 2, 100), z, w)
        dn = gdn.fused_gated_rms_norm_checkpoint_bwd(y8, z8, w, dy.view(1, T, 2, 100), workspace=ws)
        gr = gdn.gated_linear_recurrence_bwd(x, g, y, dn[0].view(1, T, D), b, cu_seqlens=cu, workspace=ws)
        return [y, f, o, *y8, *dn, *gr[:3]]

    def second():
        y, _ = gdn.gated_linear_recurrence(dy, g, cu_seqlens=cu, state_pool=pool, state_indices=idx, workspace=ws)
        gdn.state_cache_write(pool, idx, codes, scales, idx)
        gdn.state_cache_read(codes, scales, idx, pool, idx)
        s = gdn.gated_linear_recurrence_steps(x[:, :6].view(3, 2, D), g[:, :6].view(3, 2, D), pool, idx)
        return [y, s, pool, codes]

    start = pool.clone()
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for f in (first, second):
            f()
            side.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                outs = f()
            graphs.append((f, gr, outs))
    torch.cuda.synchronize()
    for turn in range(4):
        for t in (x, dy, h0):
            t.copy_(torch.randn(t.shape, generator=d.gen).to(t.dtype))
        for f, gr, outs in graphs if turn % 2 else graphs[::-1]:
            pool.copy_(start)
            want = [t.clone() for t in f()]
            ws.fill_(turn)
            pool.copy_(start)
            gr.replay()
            torch.cuda.synchronize()
            for i, (a, e) in enumerate(zip(outs, want)):
                assert torch.equal(a, e), (turn, f.__name__, i)


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, give the bits of calls one after the other."""
    gdn = _gdn()
    d = Draw(9)
    sets = [(d.randn(1, 5000, 260, dtype=BF), d.gates(1, 5000, 260, dtype=t), d.rand(1, 5000, 260, dtype=t)) for t in (F32, BF)]
    want = [gdn.gated_linear_recurrence(*s) for s in sets]
    grads = [gdn.gated_linear_recurrence_bwd(s[0], s[1], w[0], s[0], s[2]) for s, w in zip(sets, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for st, s, w, o in zip(streams, sets, want, got):
            with torch.cuda.stream(st):
                o.append(gdn.gated_linear_recurrence(*s) + gdn.gated_linear_recurrence_bwd(s[0], s[1], w[0], s[0], s[2])[:3])
    torch.cuda.synchronize()
    for o, w, gr in zip(got, want, grads):
        for r in o:
            assert all(torch.equal(a, e) for a, e in zip(r, w + gr[:3]))


def test_a_slot_named_twice_ends_with_the_later_token():
    gdn = _gdn()
    d = Draw(10)
    x, g = d.randn(2, 3, 50), d.gates(2, 3, 50)
    pool = d.randn(4, 50)
    idx = torch.tensor([[2, 2, 1], [0, 3, 3]], dtype=I32, device=DEV)
    ref, _, _, _ = orc.scan(x, g, None, pool[[2, 0]])
    gdn.gated_linear_recurrence_steps(x, g, pool, idx)
    for slot, row, tok in ((2, 0, 1), (1, 0, 2), (0, 1, 0), (3, 1, 2)):
        np.testing.assert_allclose(_np(pool[slot]), ref[row, tok], rtol=1e-5, atol=1e-5)


def test_rows_of_one_stride_and_off_alignment():
    """Inputs that are parts of wider rows, begin off alignment or repeat with stride 0 give the bits of their copies."""
    gdn = _gdn()
    d = Draw(11)
    B, T, D = 2, 150, 45
    for dtype, gate in ((BF, BF), (BF, F32), (F32, F32)):
        wide, wg = d.randn(B, T, 3 * D + 1, dtype=dtype), d.gates(B, T, 2 * D + 3, dtype=gate)
        x, g, b = wide[..., D + 1:2 * D + 1], wg[..., 1:D + 1], wg[..., D + 2:2 * D + 2]
        dy, y = d.randn(B, T, D, dtype=dtype), d.randn(B, T, D, dtype=dtype)
        copies = [t.clone(memory_format=torch.contiguous_format) for t in (x, g, b)]
        for u, v in zip(gdn.gated_linear_recurrence(x, g, b), gdn.gated_linear_recurrence(*copies)):
            assert torch.equal(u, v)
        one = gdn.gated_linear_recurrence_bwd(x, g, y, dy, b)
        two = gdn.gated_linear_recurrence_bwd(copies[0], copies[1], y, dy, copies[2])
        assert all(torch.equal(u, v) for u, v in zip(one[:3], two[:3]))
        rep, same = x[:, :1].expand(B, T, D), x[:, :1].expand(B, T, D).contiguous()
        assert torch.equal(gdn.gated_linear_recurrence(rep, g)[0], gdn.gated_linear_recurrence(same, g)[0])
        assert torch.equal(gdn.checkpoint_activation(rep).codes, gdn.checkpoint_activation(same).codes)
        turned = x.transpose(0, 1)
        assert torch.equal(gdn.checkpoint_activation(turned).codes, gdn.checkpoint_activation(turned.contiguous()).codes)


def test_calls_without_tokens():
    gdn = _gdn()
    h = torch.randn(2, 6, device=DEV)
    e = torch.zeros(2, 0, 6, device=DEV)
    y, f = gdn.gated_linear_recurrence(e, e, initial_state=h)
    assert y.shape == e.shape and torch.equal(f, h)
    dx, dg, db, dh = gdn.gated_linear_recurrence_bwd(None, e, e, e, dht=h, output_dinitial=True)
    assert torch.equal(dh, h) and db is None and dx.shape == e.shape
    _, f = gdn.gated_linear_recurrence(e, e)
    assert not f.any()
    pool = torch.ones(3, 6, device=DEV)
    idx = torch.tensor([2, 7], dtype=I32, device=DEV)
    gdn.gated_linear_recurrence(e, e, state_pool=pool, state_indices=idx)
    assert (pool == 1).all()
    gdn.gated_linear_recurrence(e, e, state_pool=pool, state_indices=idx, read_initial_state=False)
    assert (pool[:2] == 1).all() and not pool[2].any()
    none = torch.zeros(0, 4, 6, device=DEV)
    y, f = gdn.gated_linear_recurrence(none, none)
    assert y.shape == none.shape and f.shape == (0, 6)
    c = gdn.checkpoint_activation(none)
    assert c.codes.shape == none.shape and gdn.restore_activation(c).shape == none.shape
    out, cx, cz = gdn.fused_gated_rms_norm_checkpoint(none, none, torch.ones(6, device=DEV))
    dx, dz, dw = gdn.fused_gated_rms_norm_checkpoint_bwd(cx, cz, torch.ones(6, device=DEV), none)
    assert not dw.any() and dx.shape == none.shape
    codes, scales = gdn.make_state_cache(pool, 2)
    gdn.state_cache_write(pool, idx[:0], codes, scales, idx[:0])
    assert not codes.any()
