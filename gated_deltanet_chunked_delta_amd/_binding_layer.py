"""ctypes binding of the operators around the delta rule in include/gdn.h: the
recurrent steps over several tokens, the short causal convolution and the RMS
norms, forward and backward.

As in ``_binding``: argument marshalling only, no CPU path.  These calls are
short on a decode batch, so the wrappers keep their own work small: plain
integers instead of ctypes objects, one struct per call.  A call on another
device than the current one makes that device current for its duration.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from ._binding import _DTYPES, GDN_OK, GdnError, _check, _gate_inputs, gdn_gates, gdn_shape, gdn_state_pool

EXPORTED_LAYER = ("gdn_recurrent_steps", "gdn_conv_fwd", "gdn_conv_fwd_pool", "gdn_conv_update", "gdn_conv_bwd",
                  "gdn_conv_bwd_workspace_bytes", "gdn_gated_norm", "gdn_gated_norm_bwd", "gdn_add_norm",
                  "gdn_add_norm_bwd", "gdn_norm_bwd_workspace_bytes")


class gdn_step_pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("indices", ctypes.c_void_p), ("num_accepted", ctypes.c_void_p),
                ("pool_size", ctypes.c_int32), ("cols", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class gdn_conv_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32), ("W", ctypes.c_int32),
                ("N", ctypes.c_int32), ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("x_stride", ctypes.c_int64)]


class gdn_conv_pieces(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p * 3), ("dim", ctypes.c_int32 * 3)]


class gdn_norm_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("z_stride", ctypes.c_int64), ("D", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32)]


_lib = None


def _load():
    """libgdn.so with the signatures of these entry points declared."""
    global _lib
    if _lib is None:
        lib = _b.load_library()
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        sigs = {
            "gdn_recurrent_steps": (I, [P, P, P, P, P, P, F, I, P, P, P, P, P]),
            "gdn_conv_fwd": (I, [P, P, P, I, P, P, P, P, P, P]),
            "gdn_conv_fwd_pool": (I, [P, P, P, I, P, P, P, P, P]),
            "gdn_conv_update": (I, [P, P, P, I, P, P, P, P, P]),
            "gdn_conv_bwd": (I, [P, P, P, I, P, P, P, P, P, P, P, P, P, Z, P]),
            "gdn_conv_bwd_workspace_bytes": (Z, [P]),
            "gdn_gated_norm": (I, [P, P, P, F, P, P, P]),
            "gdn_gated_norm_bwd": (I, [P, P, P, F, P, P, P, P, P, P, Z, P]),
            "gdn_add_norm": (I, [P, P, P, F, F, F, P, P, P, P]),
            "gdn_add_norm_bwd": (I, [P, P, P, P, F, F, F, P, P, P, P, P, Z, P]),
            "gdn_norm_bwd_workspace_bytes": (Z, [P]),
        }
        for name, (res, args) in sigs.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib = lib
    return _lib


def _p(t):
    return None if t is None else t.data_ptr()


def _r(s):
    return None if s is None else ctypes.addressof(s)


def _stream_of(t, stream):
    return torch.cuda.current_stream(t.device).cuda_stream if stream is None else int(stream)


def _bytes(t, nbytes):
    return nbytes if nbytes is not None else 0 if t is None else t.numel() * t.element_size()


# ---------------------------------------------------------------------------
# Direct calls of the C entry points: each returns the status code.  `stream`
# is a raw hipStream_t handle or None for torch's current stream.
# ---------------------------------------------------------------------------
def gdn_recurrent_steps(q, k, v, g, beta, gates, scale, use_l2norm, pool: gdn_step_pool, cu_seqlens, out,
                        shape: gdn_shape, stream=None) -> int:
    return _load().gdn_recurrent_steps(_p(q), _p(k), _p(v), _p(g), _p(beta), _r(gates), scale, bool(use_l2norm),
                                       _r(pool), _p(cu_seqlens), _p(out), _r(shape), _stream_of(q, stream))


def gdn_conv_fwd(x, weight, bias, silu, initial_state, cu_seqlens, out: gdn_conv_pieces, final_state,
                 shape: gdn_conv_shape, stream=None) -> int:
    return _load().gdn_conv_fwd(_p(x), _p(weight), _p(bias), bool(silu), _p(initial_state), _p(cu_seqlens), _r(out),
                                _p(final_state), _r(shape), _stream_of(x, stream))


def gdn_conv_fwd_pool(x, weight, bias, silu, pool: gdn_state_pool, cu_seqlens, out: gdn_conv_pieces,
                      shape: gdn_conv_shape, stream=None) -> int:
    return _load().gdn_conv_fwd_pool(_p(x), _p(weight), _p(bias), bool(silu), _r(pool), _p(cu_seqlens), _r(out),
                                     _r(shape), _stream_of(x, stream))


def gdn_conv_update(x, weight, bias, silu, pool: gdn_step_pool, cu_seqlens, out: gdn_conv_pieces,
                    shape: gdn_conv_shape, stream=None) -> int:
    return _load().gdn_conv_update(_p(x), _p(weight), _p(bias), bool(silu), _r(pool), _p(cu_seqlens), _r(out),
                                   _r(shape), _stream_of(x, stream))


def gdn_conv_bwd_workspace_bytes(shape: gdn_conv_shape) -> int:
    return _load().gdn_conv_bwd_workspace_bytes(_r(shape))


def gdn_conv_bwd(x, weight, bias, silu, initial_state, cu_seqlens, dout: gdn_conv_pieces, dx, dweight, dbias,
                 dinitial, shape: gdn_conv_shape, workspace, workspace_bytes=None, stream=None) -> int:
    return _load().gdn_conv_bwd(_p(x), _p(weight), _p(bias), bool(silu), _p(initial_state), _p(cu_seqlens), _r(dout),
                                _p(dx), _p(dweight), _p(dbias), _p(dinitial), _r(shape), _p(workspace),
                                _bytes(workspace, workspace_bytes), _stream_of(x, stream))


def gdn_gated_norm(x, z, weight, eps, out, shape: gdn_norm_shape, stream=None) -> int:
    return _load().gdn_gated_norm(_p(x), _p(z), _p(weight), eps, _p(out), _r(shape), _stream_of(x, stream))


def gdn_gated_norm_bwd(x, z, weight, eps, dout, dx, dz, dweight, shape: gdn_norm_shape, workspace,
                       workspace_bytes=None, stream=None) -> int:
    return _load().gdn_gated_norm_bwd(_p(x), _p(z), _p(weight), eps, _p(dout), _p(dx), _p(dz), _p(dweight), _r(shape),
                                      _p(workspace), _bytes(workspace, workspace_bytes), _stream_of(x, stream))


def gdn_add_norm(x, residual, weight, residual_scale, weight_offset, eps, out, hidden, shape: gdn_norm_shape,
                 stream=None) -> int:
    return _load().gdn_add_norm(_p(x), _p(residual), _p(weight), residual_scale, weight_offset, eps, _p(out),
                                _p(hidden), _r(shape), _stream_of(x, stream))


def gdn_norm_bwd_workspace_bytes(shape: gdn_norm_shape) -> int:
    return _load().gdn_norm_bwd_workspace_bytes(_r(shape))


def gdn_add_norm_bwd(dout, dhidden, hidden, weight, residual_scale, weight_offset, eps, dx, dresidual, dweight,
                     shape: gdn_norm_shape, workspace, workspace_bytes=None, stream=None) -> int:
    return _load().gdn_add_norm_bwd(_p(dout), _p(dhidden), _p(hidden), _p(weight), residual_scale, weight_offset, eps,
                                    _p(dx), _p(dresidual), _p(dweight), _r(shape), _p(workspace),
                                    _bytes(workspace, workspace_bytes), _stream_of(dout, stream))


def _call(fn, *args):
    """fn(*args) with its first tensor's device current; raises on a bad status."""
    dev = args[0].device
    if dev.index == torch.cuda.current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != GDN_OK:
        raise GdnError(st)


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}")


def _weight_dtype(x, weight, name):
    _check(weight.dtype == x.dtype or weight.dtype == torch.float32, f"{name} must be {x.dtype} or float32")
    return _DTYPES[weight.dtype]


def make_step_pool(data, indices, num_accepted=None) -> gdn_step_pool:
    """A gdn_step_pool struct over [P, ...] slots and [N, cols] (or [N]) int32
    indices (the tensors must stay alive while it is used)."""
    return gdn_step_pool(data.data_ptr(), indices.data_ptr(), _p(num_accepted), data.shape[0],
                         indices.shape[1] if indices.dim() == 2 else 1, _DTYPES[data.dtype])


def _step_pool(data, indices, num_accepted, N, dev, slot, name):
    """Checks a few-token step's pool, indices [N] or [N, cols] and accepted counts."""
    _check(data.dim() == 1 + len(slot) and tuple(data.shape[1:]) == slot and data.is_contiguous(),
           f"{name} must be a contiguous [P,{','.join(map(str, slot))}]")
    _check(indices.dtype == torch.int32 and indices.dim() in (1, 2) and indices.shape[0] == N
           and (indices.dim() == 1 or indices.shape[1] > 0), f"{name}'s indices must be int32 [{N}] or [{N},cols]")
    _check(num_accepted is None or (num_accepted.dtype == torch.int32 and tuple(num_accepted.shape) == (N,)),
           f"num_accepted must be int32 [{N}]")
    _same_device(dev, pool=data, indices=indices, num_accepted=num_accepted)


def _sequences(x, cu_seqlens):
    """Number of sequences of x [B, T, ...]."""
    if cu_seqlens is None:
        return x.shape[0]
    _check(x.shape[0] == 1, "cu_seqlens requires B == 1")
    _check(cu_seqlens.dim() == 1 and cu_seqlens.dtype == torch.int32 and cu_seqlens.shape[0] > 0,
           "cu_seqlens must be int32 [N+1]")
    _check(cu_seqlens.device == x.device, f"cu_seqlens must be on {x.device}")
    return cu_seqlens.shape[0] - 1


def fused_recurrent_gated_delta_rule_steps(q, k, v, g, beta, state_pool, state_indices, cu_seqlens=None,
                                           num_accepted=None, scale=None, use_qk_l2norm_in_kernel=False, out=None,
                                           A_log=None, dt_bias=None, a_raw=None, b_raw=None):
    """The gated delta rule over a few tokens per sequence, states in a pool.

    q, k [B,T,H,K], v [B,T,HV,V] (bf16, or fp32 for the check mode), one
    sequence per row, or B = 1 and ``cu_seqlens`` [N+1] int32; g, beta [B,T,HV]
    fp32, or None with the raw gate inputs A_log, dt_bias [HV] fp32 and a_raw,
    b_raw [B,T,HV] (q's dtype).  state_pool [P,HV,K,V] float32 or bfloat16 is
    updated in place; state_indices int32 [N] (one slot per sequence) or
    [N,cols].  Sequence n starts from slot state_indices[n, num_accepted[n] - 1]
    (column 0 without ``num_accepted``, int32 [N], taken into [1, cols]); column
    c < cols - 1 then holds the state after its token c + 1, the last column the
    state after its last token.  A start slot outside [0, P) marks a padding
    row: zeros in the output, nothing stored.  Returns o with v's shape.
    """
    _check(q.dim() == 4 and k.shape == q.shape, "q and k must be [B,T,H,K] of equal shape")
    B, T, H, K = q.shape
    _check(v.dim() == 4 and v.shape[0] == B and v.shape[1] == T, "v must be [B,T,HV,V]")
    HV, V = v.shape[2], v.shape[3]
    dt = q.dtype
    _check(dt in _DTYPES and k.dtype == dt and v.dtype == dt, "q, k, v must share one dtype (bfloat16 or float32)")
    _check(q.is_cuda, "tensors must be on a GPU device (there is no CPU path)")
    dev = q.device
    N = _sequences(q, cu_seqlens)
    gates = None
    if g is None and beta is None:
        A_log, dt_bias, a_raw, b_raw = _gate_inputs(A_log, dt_bias, a_raw, b_raw, (B, T, HV), dt, dev)
        gates = gdn_gates(A_log.data_ptr(), dt_bias.data_ptr(), a_raw.data_ptr(), b_raw.data_ptr())
    else:
        _check(g is not None and beta is not None and A_log is None and dt_bias is None and a_raw is None
               and b_raw is None, "give either g and beta or the raw gate inputs")
        _check(tuple(g.shape) == (B, T, HV) and g.dtype == torch.float32, "g must be float32 [B,T,HV]")
        _check(tuple(beta.shape) == (B, T, HV) and beta.dtype == torch.float32, "beta must be float32 [B,T,HV]")
        _same_device(dev, g=g, beta=beta)
        g, beta = g.contiguous(), beta.contiguous()
    _same_device(dev, k=k, v=v)
    _check(state_pool.dtype in _DTYPES, "state_pool must be float32 or bfloat16")
    _step_pool(state_pool, state_indices, num_accepted, N, dev, (HV, K, V), "state_pool")
    if out is None:
        out = torch.empty((B, T, HV, V), dtype=dt, device=dev)
    else:
        _check(out.shape == v.shape and out.dtype == dt and out.is_contiguous() and out.device == dev,
               f"out must be a contiguous {dt} [{B},{T},{HV},{V}] on {dev}")
    idx = state_indices.contiguous()
    acc = None if num_accepted is None else num_accepted.contiguous()
    cu = None if cu_seqlens is None else cu_seqlens.contiguous()
    _call(gdn_recurrent_steps, q.contiguous(), k.contiguous(), v.contiguous(), g, beta, gates,
          K ** -0.5 if scale is None else float(scale), use_qk_l2norm_in_kernel, make_step_pool(state_pool, idx, acc),
          cu, out, gdn_shape(B, T, H, HV, K, V, N, _DTYPES[dt]))
    return out


# ---------------------------------------------------------------------------
# Short convolution
# ---------------------------------------------------------------------------
def _row_stride(x):
    """x [B, T, D] as rows of one stride: (x or a contiguous copy, stride)."""
    B, T, D = x.shape
    if not x.is_contiguous():
        sb, st, sd = x.stride()
        rs = st if T > 1 else sb if B > 1 else D
        if (sd == 1 or D == 1) and D <= rs <= 1 << 31 and (T == 1 or B == 1 or sb == T * rs):
            return x, rs
        x = x.contiguous()
    return x, D


def _conv_args(x, weight, bias, cu_seqlens, activation):
    _check(x.dim() == 3 and x.dtype in _DTYPES, "x must be bfloat16 or float32 [B,T,D]")
    _check(x.is_cuda, "tensors must be on a GPU device (there is no CPU path)")
    B, T, D = x.shape
    _check(weight.dim() == 2 and weight.shape[0] == D, f"weight must be [{D},W]")
    wd = _weight_dtype(x, weight, "weight")
    _check(bias is None or (tuple(bias.shape) == (D,) and bias.dtype == weight.dtype),
           f"bias must be {weight.dtype} [{D}]")
    _check(activation in ("silu", "swish", None), 'activation must be "silu" (or "swish") or None')
    _same_device(x.device, weight=weight, bias=bias)
    N = _sequences(x, cu_seqlens)
    xr, rs = _row_stride(x)
    shape = gdn_conv_shape(B, T, D, weight.shape[1], N, _DTYPES[x.dtype], wd, max(rs, D))
    return (xr, weight.contiguous(), None if bias is None else bias.contiguous(),
            None if cu_seqlens is None else cu_seqlens.contiguous(), shape, N, activation is not None)


def _conv_out(x, split_sizes, out, name="out"):
    """The output tensors: given or new, one or one per split size; and their struct."""
    B, T, D = x.shape
    sizes = (D,) if split_sizes is None else tuple(split_sizes)
    _check(1 <= len(sizes) <= 3 and min(sizes) >= 0 and sum(sizes) == D,
           f"split_sizes must be one to three sizes that sum to {D}")
    if out is None:
        outs = [torch.empty((B, T, n), dtype=x.dtype, device=x.device) for n in sizes]
    else:
        outs = [out] if isinstance(out, torch.Tensor) else list(out)
        _check(len(outs) == len(sizes), f"{name} must be one tensor per split size")
        for t, n in zip(outs, sizes):
            _check(tuple(t.shape) == (B, T, n) and t.dtype == x.dtype and t.is_contiguous() and t.device == x.device,
                   f"{name} must be contiguous {x.dtype} [{B},{T},{n}] on {x.device}")
    pieces = gdn_conv_pieces()
    for i, t in enumerate(outs):
        pieces.ptr[i], pieces.dim[i] = t.data_ptr(), sizes[i]
    return outs, pieces


def causal_conv1d(x, weight, bias=None, initial_state=None, output_final_state=True, cu_seqlens=None,
                  activation="silu", split_sizes=None, out=None, final_state=None, conv_state_pool=None,
                  conv_state_indices=None, read_initial_state=True):
    """Causal depthwise convolution over the last W tokens with SiLU.

    x [B,T,D] (bf16 or fp32; its rows may be a part of wider ones), one sequence
    per row, or B = 1 and ``cu_seqlens`` [N+1] int32; weight [D,W], W = 2, 3 or
    4, and bias [D] or None in x's dtype or float32; ``activation`` "silu" or
    None.  initial_state [N,D,W-1] in x's dtype holds the inputs before each
    sequence, oldest first (None = zeros).  Returns ``(y, final_state)``: y
    [B,T,D], or with ``split_sizes`` (up to three, summing to D) a tuple of
    contiguous [B,T,size] tensors, ready as q, k and v; final_state [N,D,W-1] or
    None.  ``out`` and ``final_state`` (which may be initial_state) are used as
    given.

    With ``conv_state_pool`` [P,D,W-1] and ``conv_state_indices`` [N] int32,
    sequence n starts from slot conv_state_indices[n] (from zeros if
    ``read_initial_state`` is False or the slot is outside the pool) and leaves
    its final state there; the call then returns ``(y, None)``.
    """
    xr, w, b, cu, shape, N, silu = _conv_args(x, weight, bias, cu_seqlens, activation)
    slot = (x.shape[2], shape.W - 1)
    outs, pieces = _conv_out(x, split_sizes, out)
    y = outs[0] if split_sizes is None else tuple(outs)
    if conv_state_pool is not None:
        _check(initial_state is None and final_state is None,
               "with a state pool, initial and final states live in the pool")
        _check(conv_state_pool.dtype == x.dtype, f"conv_state_pool must be {x.dtype}")
        _check(conv_state_indices is not None and conv_state_indices.dim() == 1, f"conv_state_indices must be int32 [{N}]")
        _step_pool(conv_state_pool, conv_state_indices, None, N, x.device, slot, "conv_state_pool")
        idx = conv_state_indices.contiguous()
        _call(gdn_conv_fwd_pool, xr, w, b, silu, _b.make_state_pool(conv_state_pool, idx, read_initial_state), cu,
              pieces, shape)
        return y, None
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        _check(t is None or (tuple(t.shape) == (N, *slot) and t.dtype == x.dtype and t.device == x.device),
               f"{name} must be {x.dtype} [{N},{slot[0]},{slot[1]}] on {x.device}")
    _check(final_state is None or final_state.is_contiguous(), "final_state must be contiguous")
    if initial_state is not None:
        initial_state = initial_state.contiguous()
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = torch.empty((N, *slot), dtype=x.dtype, device=x.device)
    _call(gdn_conv_fwd, xr, w, b, silu, initial_state, cu, pieces, final_state, shape)
    return y, final_state


def causal_conv1d_update(x, weight, conv_state_pool, conv_state_indices, bias=None, cu_seqlens=None,
                         num_accepted=None, activation="silu", split_sizes=None, out=None):
    """The convolution of a few tokens per sequence, histories in a pool.

    x [N,D] (one token each), [N,T,D], or [1,T,D] with ``cu_seqlens``; weight,
    bias, activation and split_sizes as for causal_conv1d; conv_state_pool
    [P,D,W-1] in x's dtype, updated in place; conv_state_indices int32 [N] or
    [N,cols] and ``num_accepted`` as for fused_recurrent_gated_delta_rule_steps:
    the start slot, the slots that keep the history after each token, and padding
    rows (zeros, nothing stored).  Returns y with x's shape, or a tuple of
    [..., size] tensors.
    """
    flat = x.dim() == 2
    if flat:
        _check(cu_seqlens is None, "x [N,D] takes one token per sequence")
        x = x.unsqueeze(1)
    xr, w, b, cu, shape, N, silu = _conv_args(x, weight, bias, cu_seqlens, activation)
    _check(conv_state_pool.dtype == x.dtype, f"conv_state_pool must be {x.dtype}")
    _step_pool(conv_state_pool, conv_state_indices, num_accepted, N, x.device, (x.shape[2], shape.W - 1),
               "conv_state_pool")
    if flat and out is not None:
        out = out.unsqueeze(1) if isinstance(out, torch.Tensor) else [t.unsqueeze(1) for t in out]
    outs, pieces = _conv_out(x, split_sizes, out)
    idx = conv_state_indices.contiguous()
    acc = None if num_accepted is None else num_accepted.contiguous()
    _call(gdn_conv_update, xr, w, b, silu, make_step_pool(conv_state_pool, idx, acc), cu, pieces, shape)
    if flat:
        outs = [t.squeeze(1) for t in outs]
    return outs[0] if split_sizes is None else tuple(outs)


def causal_conv1d_bwd(x, weight, dy, bias=None, initial_state=None, cu_seqlens=None, activation="silu",
                      output_dinitial=False, workspace=None):
    """Backward pass of ``causal_conv1d`` (without a pool).

    ``dy``: the gradient of y, one tensor [B,T,D] or the tuple of its parts.
    Returns ``(dx, dweight, dbias, dinitial)``: dx [B,T,D] in x's dtype, dweight
    [D,W] and dbias [D] float32 (None without bias), dinitial [N,D,W-1] in x's
    dtype (None unless ``output_dinitial``).  A preallocated uint8 ``workspace``
    of gdn_conv_bwd_workspace_bytes bytes may be given.
    """
    xr, w, b, cu, shape, N, silu = _conv_args(x, weight, bias, cu_seqlens, activation)
    B, T, D = x.shape
    dev = x.device
    dys = [dy] if isinstance(dy, torch.Tensor) else list(dy)
    _check(all(t.dim() == 3 and t.dtype == x.dtype for t in dys), "dy must have x's dtype and [B,T,...] shapes")
    dys = [t.contiguous() for t in dys]
    _, pieces = _conv_out(x, [t.shape[2] for t in dys], dys, "dy")
    slot = (N, D, shape.W - 1)
    if initial_state is not None:
        _check(tuple(initial_state.shape) == slot and initial_state.dtype == x.dtype and initial_state.device == dev,
               f"initial_state must be {x.dtype} [{slot[0]},{slot[1]},{slot[2]}] on {dev}")
        initial_state = initial_state.contiguous()
    need = gdn_conv_bwd_workspace_bytes(shape)
    if workspace is None or _bytes(workspace, None) < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    else:
        _check(workspace.device == dev and workspace.is_contiguous(), f"workspace must be a contiguous buffer on {dev}")
    dx = torch.empty((B, T, D), dtype=x.dtype, device=dev)
    dweight = torch.empty((D, shape.W), dtype=torch.float32, device=dev)
    dbias = None if bias is None else torch.empty(D, dtype=torch.float32, device=dev)
    dinitial = torch.empty(slot, dtype=x.dtype, device=dev) if output_dinitial else None
    _call(gdn_conv_bwd, xr, w, b, silu, initial_state, cu, pieces, dx, dweight, dbias, dinitial, shape, workspace)
    return dx, dweight, dbias, dinitial


# ---------------------------------------------------------------------------
# RMS norms
# ---------------------------------------------------------------------------
def _norm_args(x, weight):
    _check(x.dim() >= 1 and x.dtype in _DTYPES, "x must be bfloat16 or float32 [...,D]")
    _check(x.is_cuda, "tensors must be on a GPU device (there is no CPU path)")
    D = x.shape[-1]
    _check(weight.dim() == 1 and weight.shape[0] == D, f"weight must be [{D}]")
    _check(weight.device == x.device, f"weight must be on {x.device}")
    return gdn_norm_shape(x.numel() // D if D else 0, D, D, 1, _DTYPES[x.dtype], _weight_dtype(x, weight, "weight"))


def _like(x, **tensors):
    for name, t in tensors.items():
        _check(t is None or (t.shape == x.shape and t.dtype == x.dtype and t.device == x.device),
               f"{name} must have x's shape, dtype and device")


def _into(t, x, name):
    """An output buffer: the caller's, or a new one."""
    if t is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _like(x, **{name: t})
    _check(t.is_contiguous(), f"{name} must be contiguous")
    return t


def _gate_rows(z, shape):
    """z [..., heads, D] as tokens of heads rows with one stride between them;
    fills in shape, returns z or a contiguous copy."""
    if z.is_contiguous():
        return z
    D, dims, st = z.shape[-1], z.shape, z.stride()
    if z.dim() >= 3 and (st[-1] == 1 or D == 1) and (st[-2] == D or dims[-2] == 1):
        heads, lead = dims[-2], z.dim() - 3
    elif z.dim() == 2 and (st[-1] == 1 or D == 1):
        heads, lead = 1, 0
    else:
        return z.contiguous()
    zs = st[lead]
    for i in range(lead):
        if dims[i] != 1 and st[i] != zs * _prod(dims[i + 1:lead + 1]):
            return z.contiguous()
    if not heads * D <= zs <= 1 << 31:
        return z.contiguous()
    shape.heads, shape.z_stride = heads, zs
    return z


def _prod(dims):
    n = 1
    for d in dims:
        n *= d
    return n


def fused_gated_rms_norm(x, z, weight, eps=1e-6, out=None):
    """RMS norm of x over its last dimension, times weight and SiLU(z).

    x, z [..., D] of one shape and dtype (bf16 or fp32, D up to 1024), as the
    delta rule's output [B,T,HV,V] and its gate, which may be a part of a wider
    projection's rows; weight [D] in x's dtype or float32.  Returns x's shape."""
    shape = _norm_args(x, weight)
    _like(x, z=z)
    out = _into(out, x, "out")
    _call(gdn_gated_norm, x.contiguous(), _gate_rows(z, shape), weight.contiguous(), float(eps), out, shape)
    return out


def _norm_workspace(workspace, shape, dev):
    need = gdn_norm_bwd_workspace_bytes(shape)
    if workspace is None or _bytes(workspace, None) < need:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(workspace.device == dev and workspace.is_contiguous(), f"workspace must be a contiguous buffer on {dev}")
    return workspace


def fused_gated_rms_norm_bwd(x, z, weight, dy, eps=1e-6, workspace=None):
    """Backward pass of ``fused_gated_rms_norm``: ``(dx, dz, dweight)``, dx and
    dz in x's dtype and shape, dweight float32 [D].  A preallocated uint8
    ``workspace`` of gdn_norm_bwd_workspace_bytes bytes may be given."""
    shape = _norm_args(x, weight)
    _like(x, z=z, dy=dy)
    dev = x.device
    dx, dz = _into(None, x, "dx"), _into(None, x, "dz")
    dweight = torch.empty(x.shape[-1], dtype=torch.float32, device=dev)
    zr = _gate_rows(z, shape)
    _call(gdn_gated_norm_bwd, x.contiguous(), zr, weight.contiguous(), float(eps), dy.contiguous(), dx, dz, dweight,
          shape, _norm_workspace(workspace, shape, dev))
    return dx, dz, dweight


def fused_add_rms_norm(x, residual, weight, eps=1e-6, residual_scale=1.0, weight_offset=0.0, out=None, hidden=None):
    """hidden = residual + residual_scale * x and its RMS norm.

    x, residual [..., D] of one shape and dtype (bf16 or fp32, D up to 16384);
    residual may be None (zeros).  Returns ``(y, hidden)``, y = hidden / rms *
    (weight + weight_offset), taken from the unrounded hidden.  ``hidden`` may be
    the residual itself, which is then updated in place."""
    shape = _norm_args(x, weight)
    _like(x, residual=residual)
    out = _into(out, x, "out")
    hidden = _into(hidden, x, "hidden")
    _call(gdn_add_norm, x.contiguous(), None if residual is None else residual.contiguous(), weight.contiguous(),
          float(residual_scale), float(weight_offset), float(eps), out, hidden, shape)
    return out, hidden


def fused_add_rms_norm_bwd(dy, dhidden, hidden, weight, eps=1e-6, residual_scale=1.0, weight_offset=0.0,
                           output_dx=True, workspace=None):
    """Backward pass of ``fused_add_rms_norm`` from the hidden it returned.

    ``dy`` and ``dhidden`` (or None) are the gradients of its two outputs.
    Returns ``(dx, dresidual, dweight)`` in the inputs' dtype, dweight float32
    [D]; with residual_scale 1 dx equals dresidual, and ``output_dx=False``
    leaves it out (None)."""
    shape = _norm_args(hidden, weight)
    _like(hidden, dy=dy, dhidden=dhidden)
    dev = hidden.device
    dx = _into(None, hidden, "dx") if output_dx else None
    dresidual = _into(None, hidden, "dresidual")
    dweight = torch.empty(hidden.shape[-1], dtype=torch.float32, device=dev)
    _call(gdn_add_norm_bwd, dy.contiguous(), None if dhidden is None else dhidden.contiguous(), hidden.contiguous(),
          weight.contiguous(), float(residual_scale), float(weight_offset), float(eps), dx, dresidual, dweight, shape,
          _norm_workspace(workspace, shape, dev))
    return dx, dresidual, dweight
