"""ctypes binding of the operators around the delta rule in include/gdn.h: the
recurrent steps over several tokens, the short causal convolution and the RMS
norms, forward and backward.

As in ``_binding``: argument marshalling only, no CPU path.  On a decode batch
the wrapper's own work is most of a call, so it is kept small: plain integers
instead of ctypes objects, one struct a call, messages built only when they are
raised, torch's raw stream handle (0.1 us; ``current_stream`` takes 1.9).  A
call on another device than the current one makes that device current for its
duration.

With ``cu_seqlens[N] < T`` (a batch padded to a fixed T) the rows behind the last
sequence are neither read nor written: in a new output tensor they are undefined.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from ._binding import _DTYPES, GdnError, gdn_gates, gdn_shape, gdn_state_pool

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


_addr = ctypes.addressof
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # none in a torch without GPU support


def _stream_of(t, stream):
    return _raw_stream(t.get_device()) if stream is None else int(stream)


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


def _run(dev, fn, *args):
    """fn(*args, stream) with device number dev current; raises on a bad status.
    The tensors behind the pointers in args are the caller's to keep until then."""
    if dev == torch.cuda.current_device():
        st = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    if st:
        raise GdnError(st)


def _gpu(x, name):
    """x's device number and dtype code."""
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float32")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a GPU device (there is no CPU path)")
    return dev, code


def _weight(x, weight, bias=None):
    """dtype code of weight and bias: x's dtype or float32."""
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        raise ValueError(f"weight must be {x.dtype} or float32")
    if bias is not None and bias.dtype != weight.dtype:
        raise ValueError(f"bias must be {weight.dtype}")
    return _DTYPES[weight.dtype]


def make_step_pool(data, indices, num_accepted=None) -> gdn_step_pool:
    """A gdn_step_pool struct over [P, ...] slots and [N, cols] (or [N]) int32
    indices (the tensors must stay alive while it is used)."""
    return gdn_step_pool(data.data_ptr(), indices.data_ptr(), _p(num_accepted), data.shape[0],
                         indices.shape[1] if indices.dim() == 2 else 1, _DTYPES[data.dtype])


def _step_pool(dev, data, indices, num_accepted, N, slot, name):
    """Checks a few-token step's pool, indices [N] or [N, cols] and accepted
    counts; returns the struct and what it points to."""
    dims, acc = indices.shape, None
    if data.shape[1:] != slot or not data.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [P,{','.join(map(str, slot))}]")
    if indices.dtype != torch.int32 or not 1 <= len(dims) <= 2 or dims[0] != N or dims[-1] == 0 < N:
        raise ValueError(f"{name}'s indices must be int32 [{N}] or [{N},cols]")
    if (data.shape[0] | dims[-1]) >> 31:   # sizes are 32-bit in the structs, which do not check them
        raise ValueError(f"{name}: fewer than 2^31 slots and columns are wanted")
    if num_accepted is not None:
        if num_accepted.dtype != torch.int32 or num_accepted.shape != (N,):
            raise ValueError(f"num_accepted must be int32 [{N}]")
        if num_accepted.get_device() != dev:
            raise ValueError(f"num_accepted must be on cuda:{dev}")
        num_accepted = num_accepted.contiguous()
        acc = num_accepted.data_ptr()
    if data.get_device() != dev or indices.get_device() != dev:
        raise ValueError(f"{name} and its indices must be on cuda:{dev}")
    indices = indices.contiguous()
    pool = gdn_step_pool(data.data_ptr(), indices.data_ptr(), acc, data.shape[0], dims[1] if len(dims) == 2 else 1,
                         _DTYPES[data.dtype])
    return pool, (indices, num_accepted)


def _sequences(dev, B, cu_seqlens):
    """Number of sequences in B rows."""
    if cu_seqlens is None:
        return B
    if B != 1:
        raise ValueError("cu_seqlens requires B == 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.dtype != torch.int32 or cu_seqlens.shape[0] == 0:
        raise ValueError("cu_seqlens must be int32 [N+1]")
    if cu_seqlens.get_device() != dev:
        raise ValueError(f"cu_seqlens must be on cuda:{dev}")
    if cu_seqlens.shape[0] >> 31:
        raise ValueError("cu_seqlens must have fewer than 2^31 entries")
    return cu_seqlens.shape[0] - 1


def _given(t, shape, x, dev, name):
    """Checks a buffer that the caller hands in to be written."""
    if t.shape != shape or t.dtype != x.dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous {x.dtype} {list(shape)} on cuda:{dev}")
    return t


def _span(t):
    """First byte of t and one past its last."""
    at = t.data_ptr()
    if t.is_contiguous():
        return at, at + t.nbytes
    return at, at + t.element_size() * (1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride())))


def _apart(name, written, *read, same=()):
    """Refuses tensors to be written that overlap each other, one of read, or one
    of same without being the same elements: another workgroup may not have read
    them yet."""
    spans = [_span(t) for t in read if t is not None]
    for t in written:
        a0, a1 = span = _span(t)
        for b0, b1 in spans:
            if b0 < a1 and a0 < b1:
                raise ValueError(f"{name} must not overlap an input or another output")
        spans.append(span)
        for u in same:
            if u is not None and (u.data_ptr() != a0 or not u.is_contiguous()):
                b0, b1 = _span(u)
                if b0 < a1 and a0 < b1:
                    raise ValueError(f"{name} must not overlap a part of an input")


def _workspace(workspace, need, dev, x):
    """The caller's workspace after its checks, or a new one."""
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous buffer on cuda:{dev}")
    if workspace.nbytes < need:
        raise ValueError(f"workspace must have {need} bytes")
    return workspace


# ---------------------------------------------------------------------------
# Recurrent steps
# ---------------------------------------------------------------------------
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
    row: zeros in the output, nothing stored.  Returns o with v's shape; ``out``,
    used as given, must not overlap the inputs or the pool.
    """
    dims, vdims, dt = q.shape, v.shape, q.dtype
    if len(dims) != 4 or k.shape != dims:
        raise ValueError("q and k must be [B,T,H,K] of equal shape")
    if len(vdims) != 4 or vdims[:2] != dims[:2]:
        raise ValueError("v must be [B,T,HV,V]")
    dev, code = _gpu(q, "q")
    if k.dtype != dt or v.dtype != dt:
        raise ValueError("q, k, v must share one dtype (bfloat16 or float32)")
    B, T, H, K = dims
    HV, V = vdims[2], vdims[3]
    if (B | T) >> 31:
        raise ValueError("q must be [B,T,H,K] with sizes below 2^31")
    N = _sequences(dev, B, cu_seqlens)
    gates = gp = bp = None
    if g is None and beta is None:
        if A_log is None or dt_bias is None or a_raw is None or b_raw is None:
            raise ValueError("in-kernel gating needs all of A_log, dt_bias, a_raw, b_raw")
        if A_log.shape != (HV,) or dt_bias.shape != (HV,) or A_log.dtype != torch.float32 \
                or dt_bias.dtype != torch.float32:
            raise ValueError(f"A_log and dt_bias must be float32 [{HV}]")
        if a_raw.numel() != B * T * HV or b_raw.numel() != B * T * HV or a_raw.dtype != dt or b_raw.dtype != dt:
            raise ValueError(f"a_raw and b_raw must hold [{B},{T},{HV}] elements of q's dtype")
        g, beta, A_log, dt_bias = a_raw.contiguous(), b_raw.contiguous(), A_log.contiguous(), dt_bias.contiguous()
        gates = gdn_gates(A_log.data_ptr(), dt_bias.data_ptr(), g.data_ptr(), beta.data_ptr())
        if A_log.get_device() != dev or dt_bias.get_device() != dev:
            raise ValueError(f"A_log and dt_bias must be on cuda:{dev}")
    else:
        if g is None or beta is None or not (A_log is dt_bias is a_raw is b_raw is None):
            raise ValueError("give either g and beta or the raw gate inputs")
        if g.shape != vdims[:3] or g.dtype != torch.float32 or beta.shape != vdims[:3] or beta.dtype != torch.float32:
            raise ValueError("g and beta must be float32 [B,T,HV]")
        g, beta = g.contiguous(), beta.contiguous()
        gp, bp = g.data_ptr(), beta.data_ptr()
    if not k.get_device() == v.get_device() == g.get_device() == beta.get_device() == dev:
        raise ValueError(f"k, v and the gates must be on cuda:{dev}")
    if state_pool.dtype not in _DTYPES:
        raise ValueError("state_pool must be float32 or bfloat16")
    pool, kept = _step_pool(dev, state_pool, state_indices, num_accepted, N, (HV, K, V), "state_pool")
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if out is None:
        out = torch.empty_like(v)
    else:
        _apart("out", [_given(out, vdims, v, dev, "out")], q, k, g, beta, state_pool, same=(v,))
    if cu_seqlens is not None:
        cu_seqlens = cu_seqlens.contiguous()
    shape = gdn_shape(B, T, H, HV, K, V, N, code)
    _run(dev, (_lib or _load()).gdn_recurrent_steps, q.data_ptr(), k.data_ptr(), v.data_ptr(), gp, bp, _r(gates),
         K ** -0.5 if scale is None else scale, use_qk_l2norm_in_kernel, _addr(pool), _p(cu_seqlens), out.data_ptr(),
         _addr(shape))
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
    """Checks and lays out what the convolution's calls share: the device, x's
    rows, weight, bias, cu_seqlens, the sizes, the number of sequences."""
    dims = x.shape
    if len(dims) != 3:
        raise ValueError("x must be [B,T,D]")
    dev, code = _gpu(x, "x")
    B, T, D = dims
    if (B | T | D) >> 31:
        raise ValueError("x must be [B,T,D] with sizes below 2^31")
    if weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError(f"weight must be [{D},W]")
    if bias is not None:
        if bias.shape != (D,):
            raise ValueError(f"bias must be [{D}]")
        bias = bias.contiguous()
    wcode = _weight(x, weight, bias)
    if activation not in ("silu", "swish", None):
        raise ValueError('activation must be "silu" (or "swish") or None')
    if weight.get_device() != dev or (bias is not None and bias.get_device() != dev):
        raise ValueError(f"weight and bias must be on cuda:{dev}")
    N = _sequences(dev, B, cu_seqlens)
    if cu_seqlens is not None:
        cu_seqlens = cu_seqlens.contiguous()
    rows, rs = _row_stride(x)
    weight = weight.contiguous()
    return dev, rows, weight, bias, cu_seqlens, gdn_conv_shape(B, T, D, weight.shape[1], N, code, wcode, rs), N


def _pieces(x, sizes, tensors, dev, name):
    """The output (or its gradient) as one tensor per size, given or new; and their struct."""
    B, T, D = x.shape
    if not 1 <= len(sizes) <= 3 or sum(sizes) != D or min(sizes) < 0:
        raise ValueError(f"{name}: one to three sizes that sum to {D} are wanted")
    pieces = gdn_conv_pieces()
    if tensors is None:
        tensors = []
        for i, n in enumerate(sizes):   # empty_like is the cheaper call: q and k are of one size
            tensors.append(torch.empty_like(tensors[-1]) if i and n == sizes[i - 1] else x.new_empty((B, T, n)))
    else:
        if len(tensors) != len(sizes):
            raise ValueError(f"{name} must be one tensor per split size")
        for t, n in zip(tensors, sizes):
            _given(t, (B, T, n), x, dev, name)
    ptr, dim = pieces.ptr, pieces.dim
    for i, t in enumerate(tensors):
        ptr[i], dim[i] = t.data_ptr(), sizes[i]
    return tensors, pieces


def _listed(out):
    return None if out is None else [out] if isinstance(out, torch.Tensor) else list(out)


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
    given; they must not overlap the inputs, the pool or each other.

    With ``conv_state_pool`` [P,D,W-1] and ``conv_state_indices`` [N] int32,
    sequence n starts from slot conv_state_indices[n] (from zeros if
    ``read_initial_state`` is False or the slot is outside the pool) and leaves
    its final state there; the call then returns ``(y, None)``.
    """
    dev, rows, weight, bias, cu, shape, N = _conv_args(x, weight, bias, cu_seqlens, activation)
    D, W1 = x.shape[2], shape.W - 1
    outs, pieces = _pieces(x, (D,) if split_sizes is None else split_sizes, _listed(out), dev, "out")
    y = outs[0] if split_sizes is None else tuple(outs)
    if out is not None:
        _apart("out", outs, rows, weight, bias, initial_state, conv_state_pool)
    lib = _lib or _load()
    head = (rows.data_ptr(), weight.data_ptr(), _p(bias), activation is not None)
    if conv_state_pool is not None:
        if initial_state is not None or final_state is not None:
            raise ValueError("with a state pool, initial and final states live in the pool")
        if conv_state_pool.dtype != x.dtype:
            raise ValueError(f"conv_state_pool must be {x.dtype}")
        if conv_state_indices is None or conv_state_indices.dim() != 1:
            raise ValueError(f"conv_state_indices must be int32 [{N}]")
        _, kept = _step_pool(dev, conv_state_pool, conv_state_indices, None, N, (D, W1), "conv_state_pool")
        pool = _b.make_state_pool(conv_state_pool, kept[0], read_initial_state)
        _run(dev, lib.gdn_conv_fwd_pool, *head, _addr(pool), _p(cu), _addr(pieces), _addr(shape))
        return y, None
    if initial_state is not None:
        if initial_state.shape != (N, D, W1) or initial_state.dtype != x.dtype or initial_state.get_device() != dev:
            raise ValueError(f"initial_state must be {x.dtype} [{N},{D},{W1}] on cuda:{dev}")
        initial_state = initial_state.contiguous()
    if not output_final_state:
        final_state = None
    elif final_state is not None:
        _apart("final_state", [_given(final_state, (N, D, W1), x, dev, "final_state")], rows, weight, bias, *outs,
               same=(initial_state,))
    elif initial_state is not None:
        final_state = torch.empty_like(initial_state)
    else:
        final_state = x.new_empty((N, D, W1))
    _run(dev, lib.gdn_conv_fwd, *head, _p(initial_state), _p(cu), _addr(pieces), _p(final_state), _addr(shape))
    return y, final_state


def causal_conv1d_update(x, weight, conv_state_pool, conv_state_indices, bias=None, cu_seqlens=None,
                         num_accepted=None, activation="silu", split_sizes=None, out=None):
    """The convolution of a few tokens per sequence, histories in a pool.

    x [N,D] (one token each), [N,T,D], or [1,T,D] with ``cu_seqlens``; weight,
    bias, activation and split_sizes as for causal_conv1d; conv_state_pool
    [P,D,W-1] in x's dtype, updated in place; conv_state_indices int32 [N] or
    [N,cols] and ``num_accepted`` as for fused_recurrent_gated_delta_rule_steps:
    the start slot, the slots that keep the history after each token, and padding
    rows (zeros, nothing stored).  ``out`` as for causal_conv1d.  Returns y with
    x's shape, or a tuple of [..., size] tensors.
    """
    flat = x.dim() == 2
    out = _listed(out)
    if flat:
        if cu_seqlens is not None:
            raise ValueError("x [N,D] takes one token per sequence")
        x = x.unsqueeze(1)
        out = None if out is None else [t.unsqueeze(1) for t in out]
    dev, rows, weight, bias, cu, shape, N = _conv_args(x, weight, bias, cu_seqlens, activation)
    D = x.shape[2]
    if conv_state_pool.dtype != x.dtype:
        raise ValueError(f"conv_state_pool must be {x.dtype}")
    pool, kept = _step_pool(dev, conv_state_pool, conv_state_indices, num_accepted, N, (D, shape.W - 1),
                            "conv_state_pool")
    outs, pieces = _pieces(x, (D,) if split_sizes is None else split_sizes, out, dev, "out")
    if out is not None:
        _apart("out", outs, rows, weight, bias, conv_state_pool)
    _run(dev, (_lib or _load()).gdn_conv_update, rows.data_ptr(), weight.data_ptr(), _p(bias),
         activation is not None, _addr(pool), _p(cu), _addr(pieces), _addr(shape))
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
    of gdn_conv_bwd_workspace_bytes bytes or more, 16-byte aligned, may be given.
    """
    dev, rows, weight, bias, cu, shape, N = _conv_args(x, weight, bias, cu_seqlens, activation)
    B, T, D = x.shape
    dys = [t.contiguous() for t in _listed(dy)]
    dys, pieces = _pieces(x, [t.shape[-1] for t in dys], dys, dev, "dy")
    slot = (N, D, shape.W - 1)
    if initial_state is not None:
        if initial_state.shape != slot or initial_state.dtype != x.dtype or initial_state.get_device() != dev:
            raise ValueError(f"initial_state must be {x.dtype} {list(slot)} on cuda:{dev}")
        initial_state = initial_state.contiguous()
    lib = _lib or _load()
    need = lib.gdn_conv_bwd_workspace_bytes(_addr(shape))
    ws = _workspace(workspace, need, dev, x)
    dx = x.new_empty((B, T, D))
    dweight = torch.empty_like(weight, dtype=torch.float32)
    dbias = None if bias is None else torch.empty_like(bias, dtype=torch.float32)
    dinitial = x.new_empty(slot) if output_dinitial else None
    _run(dev, lib.gdn_conv_bwd, rows.data_ptr(), weight.data_ptr(), _p(bias), activation is not None,
         _p(initial_state), _p(cu), _addr(pieces), dx.data_ptr(), dweight.data_ptr(), _p(dbias), _p(dinitial), _addr(shape),
         ws.data_ptr(), need)
    return dx, dweight, dbias, dinitial


# ---------------------------------------------------------------------------
# RMS norms
# ---------------------------------------------------------------------------
def _norm_args(x, weight):
    """x's device number, the sizes of its rows, and weight, contiguous."""
    dev, code = _gpu(x, "x")
    D = x.shape[-1] if x.dim() else 0
    if not 0 < D < 1 << 31 or weight.shape != (D,):
        raise ValueError(f"x must be [...,D] and weight [D], 0 < D < 2^31 (x {list(x.shape)}, weight {list(weight.shape)})")
    wcode = code if weight.dtype == x.dtype else _weight(x, weight)
    if weight.get_device() != dev:
        raise ValueError(f"weight must be on cuda:{dev}")
    return dev, gdn_norm_shape(x.numel() // D, D, D, 1, code, wcode), weight.contiguous()


def _same(x, t, name):
    """t contiguous, after checking it against x."""
    if t.shape != x.shape or t.dtype != x.dtype or t.get_device() != x.get_device():
        raise ValueError(f"{name} must have x's shape, dtype and device")
    return t.contiguous()


def _gate_rows(x, z, shape):
    """z [..., heads, D] as tokens of heads rows with one stride between them;
    fills in shape, returns z or a contiguous copy."""
    if z.shape != x.shape or z.dtype != x.dtype or z.get_device() != x.get_device():
        raise ValueError("z must have x's shape, dtype and device")
    if z.is_contiguous():
        return z
    dims, st = z.shape, z.stride()
    D = dims[-1]
    if len(dims) == 2:
        heads, lead = 1, 0
    elif len(dims) > 2 and (st[-2] == D or dims[-2] == 1):
        heads, lead = dims[-2], len(dims) - 3
    else:
        return z.contiguous()
    # the leading dimensions, up to `lead`, have to be one run of tokens
    zs = run = st[lead]
    for i in range(lead, 0, -1):
        run *= dims[i]
        if st[i - 1] != run:
            return z.contiguous()
    if st[-1] != 1 or not heads * D <= zs <= 1 << 31:
        return z.contiguous()
    shape.heads, shape.z_stride = heads, zs
    return z


def fused_gated_rms_norm(x, z, weight, eps=1e-6, out=None):
    """RMS norm of x over its last dimension, times weight and SiLU(z).

    x, z [..., D] of one shape and dtype (bf16 or fp32, D up to 1024), as the
    delta rule's output [B,T,HV,V] and its gate, which may be a part of a wider
    projection's rows; weight [D] in x's dtype or float32.  Returns x's shape.  A
    row whose squares sum to infinity in fp32 gives zeros, and NaN where it is
    infinite; its gradients are undefined."""
    dev, shape, weight = _norm_args(x, weight)
    z = _gate_rows(x, z, shape)
    x = x.contiguous()
    if out is None:
        out = torch.empty_like(x)
    else:
        _apart("out", [_given(out, x.shape, x, dev, "out")], weight, same=(x, z))
    _run(dev, (_lib or _load()).gdn_gated_norm, x.data_ptr(), z.data_ptr(), weight.data_ptr(), eps, out.data_ptr(),
         _addr(shape))
    return out


def fused_gated_rms_norm_bwd(x, z, weight, dy, eps=1e-6, workspace=None):
    """Backward pass of ``fused_gated_rms_norm``: ``(dx, dz, dweight)``, dx and
    dz in x's dtype and shape, dweight float32 [D].  A preallocated uint8
    ``workspace`` of gdn_norm_bwd_workspace_bytes bytes or more, 16-byte aligned,
    may be given."""
    dev, shape, weight = _norm_args(x, weight)
    z = _gate_rows(x, z, shape)
    x, dy = x.contiguous(), _same(x, dy, "dy")
    lib = _lib or _load()
    need = lib.gdn_norm_bwd_workspace_bytes(_addr(shape))
    ws = _workspace(workspace, need, dev, x)
    dx, dz = torch.empty_like(x), torch.empty_like(x)
    dweight = torch.empty_like(weight, dtype=torch.float32)
    _run(dev, lib.gdn_gated_norm_bwd, x.data_ptr(), z.data_ptr(), weight.data_ptr(), eps, dy.data_ptr(), dx.data_ptr(),
         dz.data_ptr(), dweight.data_ptr(), _addr(shape), ws.data_ptr(), need)
    return dx, dz, dweight


def fused_add_rms_norm(x, residual, weight, eps=1e-6, residual_scale=1.0, weight_offset=0.0, out=None, hidden=None):
    """hidden = residual + residual_scale * x and its RMS norm.

    x, residual [..., D] of one shape and dtype (bf16 or fp32, D up to 16384);
    residual may be None (zeros).  Returns ``(y, hidden)``, y = hidden / rms *
    (weight + weight_offset), taken from the unrounded hidden.  ``hidden`` may be
    the residual itself, which is then updated in place.  Rows whose squares sum to
    infinity as in fused_gated_rms_norm."""
    dev, shape, weight = _norm_args(x, weight)
    if residual is not None:
        residual = _same(x, residual, "residual")
    x = x.contiguous()
    given = out is not None or (hidden is not None and hidden is not residual)
    out = torch.empty_like(x) if out is None else _given(out, x.shape, x, dev, "out")
    hidden = torch.empty_like(x) if hidden is None else _given(hidden, x.shape, x, dev, "hidden")
    if given:
        _apart("out and hidden", [out, hidden], weight, same=(x, residual))
    _run(dev, (_lib or _load()).gdn_add_norm, x.data_ptr(), _p(residual), weight.data_ptr(), residual_scale,
         weight_offset, eps, out.data_ptr(), hidden.data_ptr(), _addr(shape))
    return out, hidden


def fused_add_rms_norm_bwd(dy, dhidden, hidden, weight, eps=1e-6, residual_scale=1.0, weight_offset=0.0,
                           output_dx=True, workspace=None):
    """Backward pass of ``fused_add_rms_norm`` from the hidden it returned.

    ``dy`` and ``dhidden`` (or None) are the gradients of its two outputs.
    Returns ``(dx, dresidual, dweight)`` in the inputs' dtype, dweight float32
    [D]; with residual_scale 1 dx equals dresidual, and ``output_dx=False``
    leaves it out (None).  ``workspace`` as for fused_gated_rms_norm_bwd."""
    dev, shape, weight = _norm_args(hidden, weight)
    dy = _same(hidden, dy, "dy")
    if dhidden is not None:
        dhidden = _same(hidden, dhidden, "dhidden")
    hidden = hidden.contiguous()
    lib = _lib or _load()
    need = lib.gdn_norm_bwd_workspace_bytes(_addr(shape))
    ws = _workspace(workspace, need, dev, hidden)
    dx = torch.empty_like(hidden) if output_dx else None
    dresidual = torch.empty_like(hidden)
    dweight = torch.empty_like(weight, dtype=torch.float32)
    _run(dev, lib.gdn_add_norm_bwd, dy.data_ptr(), _p(dhidden), hidden.data_ptr(), weight.data_ptr(), residual_scale,
         weight_offset, eps, _p(dx), dresidual.data_ptr(), dweight.data_ptr(), _addr(shape), ws.data_ptr(), need)
    return dx, dresidual, dweight
