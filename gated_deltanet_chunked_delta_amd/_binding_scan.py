"""ctypes binding of the gated linear recurrence and of values held in 8 and 4 bits
in include/gdn.h: the recurrence over sequences, over a few tokens and its backward
pass, caches of states, activation checkpoints and the gated norm that keeps them.

As in ``_binding_layer``: argument marshalling only, no CPU path; a call on another
device than the current one makes that device current for its duration.  With
``cu_seqlens[N] < T`` the rows behind the last sequence are neither read nor written.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _binding as _b
from . import _binding_layer as _l
from ._binding import _DTYPES, gdn_state_pool
from ._binding_layer import (_addr, _apart, _bytes, _gate_rows, _given, _gpu, _norm_args, _p, _r, _row_stride, _run,
                             _sequences, _step_pool, _stream_of, _workspace, gdn_norm_shape, gdn_step_pool)

EXPORTED_SCAN = ("gdn_scan_fwd", "gdn_scan_fwd_pool", "gdn_scan_steps", "gdn_scan_bwd", "gdn_scan_workspace_bytes",
                 "gdn_hold", "gdn_restore", "gdn_gated_norm_hold", "gdn_gated_norm_hold_bwd")

GROUP = 32   # values of one scale
_CODE_BITS = {torch.int8: 8, torch.uint8: 4}


class gdn_scan_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32), ("N", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("g_stride", ctypes.c_int64), ("beta_stride", ctypes.c_int64)]


class gdn_held(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class gdn_held_shape(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("D", ctypes.c_int64), ("stride", ctypes.c_int64),
                ("value_rows", ctypes.c_int32), ("held_rows", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("bits", ctypes.c_int32)]


class Checkpoint(NamedTuple):
    """An activation kept in 8 bits: codes int8 [..., D] and scales bfloat16
    [..., ceil(D/32)]; element i stands for codes[..., i] * scales[..., i // 32]."""
    codes: torch.Tensor
    scales: torch.Tensor


_lib = None


def _load():
    """libgdn.so with the signatures of these entry points declared."""
    global _lib
    if _lib is None:
        lib = _b.load_library()
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        sigs = {
            "gdn_scan_fwd": (I, [P, P, P, P, P, P, P, P, P, Z, P]),
            "gdn_scan_fwd_pool": (I, [P, P, P, P, P, P, P, P, Z, P]),
            "gdn_scan_steps": (I, [P, P, P, P, P, P, P, P]),
            "gdn_scan_bwd": (I, [P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]),
            "gdn_scan_workspace_bytes": (Z, [P, I]),
            "gdn_hold": (I, [P, P, P, P, P, P]),
            "gdn_restore": (I, [P, P, P, P, P, P]),
            "gdn_gated_norm_hold": (I, [P, P, P, F, P, P, P, P, P]),
            "gdn_gated_norm_hold_bwd": (I, [P, P, P, F, P, P, P, P, P, P, Z, P]),
        }
        for name, (res, args) in sigs.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib = lib
    return _lib


# ---------------------------------------------------------------------------
# Direct calls of the C entry points: each returns the status code.  `stream`
# is a raw hipStream_t handle or None for torch's current stream.
# ---------------------------------------------------------------------------
def gdn_scan_workspace_bytes(shape: gdn_scan_shape, backward=False) -> int:
    return _load().gdn_scan_workspace_bytes(_r(shape), bool(backward))


def gdn_scan_fwd(x, g, beta, initial_state, cu_seqlens, out, final_state, shape: gdn_scan_shape, workspace=None,
                 workspace_bytes=None, stream=None) -> int:
    return _load().gdn_scan_fwd(_p(x), _p(g), _p(beta), _p(initial_state), _p(cu_seqlens), _p(out), _p(final_state),
                                _r(shape), _p(workspace), _bytes(workspace, workspace_bytes), _stream_of(x, stream))


def gdn_scan_fwd_pool(x, g, beta, pool: gdn_state_pool, cu_seqlens, out, shape: gdn_scan_shape, workspace=None,
                      workspace_bytes=None, stream=None) -> int:
    return _load().gdn_scan_fwd_pool(_p(x), _p(g), _p(beta), _r(pool), _p(cu_seqlens), _p(out), _r(shape),
                                     _p(workspace), _bytes(workspace, workspace_bytes), _stream_of(x, stream))


def gdn_scan_steps(x, g, beta, pool: gdn_step_pool, cu_seqlens, out, shape: gdn_scan_shape, stream=None) -> int:
    return _load().gdn_scan_steps(_p(x), _p(g), _p(beta), _r(pool), _p(cu_seqlens), _p(out), _r(shape),
                                  _stream_of(x, stream))


def gdn_scan_bwd(x, g, beta, y, x8, y8, dout, dht, initial_state, cu_seqlens, dx, dg, dbeta, dinitial,
                 shape: gdn_scan_shape, workspace=None, workspace_bytes=None, stream=None) -> int:
    return _load().gdn_scan_bwd(_p(x), _p(g), _p(beta), _p(y), _r(x8), _r(y8), _p(dout), _p(dht), _p(initial_state),
                                _p(cu_seqlens), _p(dx), _p(dg), _p(dbeta), _p(dinitial), _r(shape), _p(workspace),
                                _bytes(workspace, workspace_bytes), _stream_of(g, stream))


def gdn_hold(values, value_index, held: gdn_held, held_index, shape: gdn_held_shape, stream=None) -> int:
    return _load().gdn_hold(_p(values), _p(value_index), _r(held), _p(held_index), _r(shape),
                            _stream_of(values, stream))


def gdn_restore(held: gdn_held, held_index, values, value_index, shape: gdn_held_shape, stream=None) -> int:
    return _load().gdn_restore(_r(held), _p(held_index), _p(values), _p(value_index), _r(shape),
                               _stream_of(values, stream))


def gdn_gated_norm_hold(x, z, weight, eps, out, x8: gdn_held, z8: gdn_held, shape: gdn_norm_shape, stream=None) -> int:
    return _load().gdn_gated_norm_hold(_p(x), _p(z), _p(weight), eps, _p(out), _r(x8), _r(z8), _r(shape),
                                       _stream_of(x, stream))


def gdn_gated_norm_hold_bwd(x8: gdn_held, z8: gdn_held, weight, eps, dout, dx, dz, dweight, shape: gdn_norm_shape,
                            workspace, workspace_bytes=None, stream=None) -> int:
    return _load().gdn_gated_norm_hold_bwd(_r(x8), _r(z8), _p(weight), eps, _p(dout), _p(dx), _p(dz), _p(dweight),
                                           _r(shape), _p(workspace), _bytes(workspace, workspace_bytes),
                                           _stream_of(dout, stream))


# ---------------------------------------------------------------------------
# Gated linear recurrence
# ---------------------------------------------------------------------------
def _gates(like, g, beta, dev):
    """g and beta as rows of one stride each, after checking them against the [B,T,D]
    dims and dtype of ``like``; their dtype code."""
    dims, dtype = like
    gdtype = g.dtype
    if g.shape != dims or (gdtype != dtype and gdtype != torch.float32):
        raise ValueError(f"g must be {list(dims)} in {dtype} or float32")
    if g.get_device() != dev or (beta is not None and beta.get_device() != dev):
        raise ValueError(f"g and beta must be on cuda:{dev}")
    gs = bs = dims[2]
    if not g.is_contiguous():
        g, gs = _row_stride(g)
    if beta is not None:
        if beta.shape != dims or beta.dtype != gdtype:
            raise ValueError(f"beta must be {list(dims)} in g's dtype")
        if not beta.is_contiguous():
            beta, bs = _row_stride(beta)
    return g, gs, beta, bs, _DTYPES[gdtype]


def _scan_args(x, g, beta, cu_seqlens):
    """Checks and lays out what the forward calls share: the device, the rows, cu_seqlens, the sizes, the number
    of sequences."""
    dims = x.shape
    if len(dims) != 3:
        raise ValueError("x must be [B,T,D]")
    dev, code = _gpu(x, "x")
    B, T, D = dims
    if (B | T | D) >> 31 or not D:
        raise ValueError("x must be [B,T,D] with sizes below 2^31 and D at least 1")
    g, gs, beta, bs, gcode = _gates((dims, x.dtype), g, beta, dev)
    N, xs = B, D
    if cu_seqlens is not None:
        N = _sequences(dev, B, cu_seqlens)
        cu_seqlens = cu_seqlens.contiguous()
    if not x.is_contiguous():
        x, xs = _row_stride(x)
    return dev, x, g, beta, cu_seqlens, gdn_scan_shape(B, T, D, N, code, gcode, xs, gs, bs), N


def _state(t, N, D, dev, name):
    """A [N,D] float32 state that is read, contiguous."""
    if t.shape != (N, D) or t.dtype != torch.float32 or t.get_device() != dev:
        raise ValueError(f"{name} must be float32 [{N},{D}] on cuda:{dev}")
    return t.contiguous()


def _scratch(workspace, need, dev, like):
    """The workspace's address, its bytes, and what keeps it alive."""
    if need == 0:
        return None, 0, None
    ws = _workspace(workspace, need, dev, like)
    return ws.data_ptr(), need, ws


def gated_linear_recurrence(x, g, beta=None, initial_state=None, output_final_state=True, cu_seqlens=None, out=None,
                            final_state=None, state_pool=None, state_indices=None, read_initial_state=True,
                            workspace=None):
    """h_t = exp(g_t) h_(t-1) + beta_t x_t per channel, y_t = h_t.

    x [B,T,D] (bf16 or fp32), one sequence per row, or B = 1 and ``cu_seqlens``
    [N+1] int32; g (log-space forget gate, <= 0) and beta (None = 1) [B,T,D] in
    x's dtype or both in float32, as fused_gdn_gating writes them.  The rows of all
    three may be parts of wider ones.  initial_state [N,D] float32 (None = zeros).
    Returns ``(y, final_state)``, y in x's dtype, final_state [N,D] float32 or
    None.  ``out`` and ``final_state`` (which may be initial_state) are used as
    given; they must not overlap the inputs, the pool or each other.

    With ``state_pool`` [P,D] (float32 or bfloat16) and ``state_indices`` [N] int32,
    sequence n starts from slot state_indices[n] (from zeros if
    ``read_initial_state`` is False or the slot is outside the pool) and leaves
    its final state there (no slot may be named twice); the call then returns
    ``(y, None)``.  A preallocated uint8 ``workspace`` of gdn_scan_workspace_bytes
    bytes or more, 16-byte aligned, may be given; calls that may run at the same
    time need their own.
    """
    dev, x, g, beta, cu, shape, N = _scan_args(x, g, beta, cu_seqlens)
    D = shape.D
    lib = _lib or _load()
    if out is None:
        y = torch.empty_like(x)          # contiguous: x is, or its rows lie apart
    else:
        y = _given(out, x.shape, x, dev, "out")
        _apart("out", [y], x, g, beta, initial_state, state_pool)
    wp, wb, ws = _scratch(workspace, lib.gdn_scan_workspace_bytes(_addr(shape), 0), dev, x)
    if state_pool is not None:
        if initial_state is not None or final_state is not None:
            raise ValueError("with a state pool, initial and final states live in the pool")
        if state_pool.dtype not in _DTYPES:
            raise ValueError("state_pool must be float32 or bfloat16")
        if state_indices is None or state_indices.dim() != 1:
            raise ValueError(f"state_indices must be int32 [{N}]")
        _, kept = _step_pool(dev, state_pool, state_indices, None, N, (D,), "state_pool")
        pool = _b.make_state_pool(state_pool, kept[0], read_initial_state)
        _run(dev, lib.gdn_scan_fwd_pool, x.data_ptr(), g.data_ptr(), _p(beta), _addr(pool), _p(cu), y.data_ptr(),
             _addr(shape), wp, wb)
        return y, None
    if initial_state is not None:
        initial_state = _state(initial_state, N, D, dev, "initial_state")
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = x.new_empty((N, D), dtype=torch.float32) if initial_state is None else torch.empty_like(initial_state)
    else:
        if final_state.shape != (N, D) or final_state.dtype != torch.float32 or not final_state.is_contiguous() \
                or final_state.get_device() != dev:
            raise ValueError(f"final_state must be a contiguous float32 [{N},{D}] on cuda:{dev}")
        _apart("final_state", [final_state], x, g, beta, y, same=(initial_state,))
    _run(dev, lib.gdn_scan_fwd, x.data_ptr(), g.data_ptr(), _p(beta), _p(initial_state), _p(cu), y.data_ptr(),
         _p(final_state), _addr(shape), wp, wb)
    return y, final_state


def gated_linear_recurrence_steps(x, g, state_pool, state_indices, beta=None, cu_seqlens=None, num_accepted=None,
                                  out=None):
    """The recurrence over a few tokens per sequence, states in a pool.

    x [N,D] (one token each), [N,T,D], or [1,T,D] with ``cu_seqlens``; g and beta
    as for gated_linear_recurrence, of x's shape; state_pool [P,D] float32 or
    bfloat16, updated in place; state_indices int32 [N] or [N,cols] and
    ``num_accepted`` as for fused_recurrent_gated_delta_rule_steps: the start slot,
    the slots that keep the state after each token, and padding rows (zeros,
    nothing stored).  Returns y with x's shape; ``out``, used as given, must not
    overlap the inputs or the pool.
    """
    flat = x.dim() == 2
    if flat:
        if cu_seqlens is not None:
            raise ValueError("x [N,D] takes one token per sequence")
        if g.dim() != 2 or (beta is not None and beta.dim() != 2):
            raise ValueError("g and beta must have x's shape")
        x, g = x.unsqueeze(1), g.unsqueeze(1)
        beta = None if beta is None else beta.unsqueeze(1)
        out = None if out is None else out.unsqueeze(1)
    dev, x, g, beta, cu, shape, N = _scan_args(x, g, beta, cu_seqlens)
    if state_pool.dtype not in _DTYPES:
        raise ValueError("state_pool must be float32 or bfloat16")
    pool, kept = _step_pool(dev, state_pool, state_indices, num_accepted, N, (shape.D,), "state_pool")
    if out is None:
        out = torch.empty_like(x)
    else:
        _apart("out", [_given(out, x.shape, x, dev, "out")], x, g, beta, state_pool)
    _run(dev, (_lib or _load()).gdn_scan_steps, x.data_ptr(), g.data_ptr(), _p(beta), _addr(pool), _p(cu),
         out.data_ptr(), _addr(shape))
    return out.squeeze(1) if flat else out


def gated_linear_recurrence_bwd(x, g, y, dy, beta=None, dht=None, initial_state=None, cu_seqlens=None,
                                output_dinitial=False, workspace=None):
    """Backward pass of ``gated_linear_recurrence`` (without a pool).

    ``y``: what the forward call returned; ``dy`` [B,T,D] its gradient, in the same
    dtype; ``dht`` [N,D] float32 that of the final state, or None.  ``x`` is read
    only with ``beta`` (it may be None without).  y, and with beta x, may instead
    be the Checkpoints of these tensors (y's may come from
    fused_gated_rms_norm_checkpoint, with y seen as [B,T,heads,dim] and dim a
    multiple of 32; other dims are refused): the gradients are then taken at the
    values that they stand for.
    Returns ``(dx, dg, dbeta, dinitial)``: dx in dy's dtype, dg and dbeta in the
    gates', dinitial [N,D] float32; dbeta is None without beta, dinitial None
    unless ``output_dinitial``.  ``workspace`` as for the forward call, of
    gdn_scan_workspace_bytes(shape, 1) bytes.
    """
    dims = dy.shape
    if len(dims) != 3:
        raise ValueError("dy must be [B,T,D]")
    dev, code = _gpu(dy, "dy")
    B, T, D = dims
    if (B | T | D) >> 31 or not D:
        raise ValueError("dy must be [B,T,D] with sizes below 2^31 and D at least 1")
    g, gs, beta, bs, gcode = _gates((dims, dy.dtype), g, beta, dev)
    N = _sequences(dev, B, cu_seqlens)
    if cu_seqlens is not None:
        cu_seqlens = cu_seqlens.contiguous()
    held = isinstance(y, Checkpoint)
    if beta is None:
        x = None
    elif x is None or held != isinstance(x, Checkpoint):
        raise ValueError("with beta, x and y must be two tensors or two checkpoints")
    x8 = y8 = None
    xs = D
    if held:
        kept, y8 = _held_rows(y, B * T, D, dev, "y")
        if x is not None:
            kept_x, x8 = _held_rows(x, B * T, D, dev, "x")
        xp = yp = None
    else:
        if y.shape != dims or y.dtype != dy.dtype or y.get_device() != dev:
            raise ValueError("y must have dy's shape, dtype and device")
        y = y.contiguous()
        if x is not None:
            if x.shape != dims or x.dtype != dy.dtype or x.get_device() != dev:
                raise ValueError("x must have dy's shape, dtype and device")
            x, xs = _row_stride(x)
        xp, yp = _p(x), y.data_ptr()
    dy = dy.contiguous()
    if dht is not None:
        dht = _state(dht, N, D, dev, "dht")
    if initial_state is not None:
        initial_state = _state(initial_state, N, D, dev, "initial_state")
    shape = gdn_scan_shape(B, T, D, N, code, gcode, xs, gs, bs)
    lib = _lib or _load()
    wp, wb, ws = _scratch(workspace, lib.gdn_scan_workspace_bytes(_addr(shape), 1), dev, dy)
    dx = torch.empty_like(dy)
    dg = torch.empty_like(dy, dtype=g.dtype)
    dbeta = None if beta is None else torch.empty_like(dg)
    dinitial = dy.new_empty((N, D), dtype=torch.float32) if output_dinitial else None
    _run(dev, lib.gdn_scan_bwd, xp, g.data_ptr(), _p(beta), yp, _r(x8), _r(y8), dy.data_ptr(), _p(dht),
         _p(initial_state), _p(cu_seqlens), dx.data_ptr(), dg.data_ptr(), _p(dbeta), _p(dinitial), _addr(shape), wp, wb)
    return dx, dg, dbeta, dinitial


# ---------------------------------------------------------------------------
# Values held in 8 and 4 bits
# ---------------------------------------------------------------------------
def _held_rows(c, rows, D, dev, name):
    """A checkpoint of rows of D values: its tensors, contiguous, and the struct."""
    codes, scales = c
    dims = codes.shape
    if codes.dtype != torch.int8 or scales.dtype != torch.bfloat16:
        raise ValueError(f"{name}: a checkpoint has int8 codes and bfloat16 scales")
    if codes.numel() != rows * D or scales.numel() != rows * -(-D // GROUP):
        raise ValueError(f"{name}: codes and scales must be those of {rows} rows of {D} values")
    if not dims or (dims[-1] != D and (D % GROUP or dims[-1] % GROUP)):
        raise ValueError(f"{name}: a checkpoint of other rows than {D} values needs both in whole groups of {GROUP}")
    if codes.get_device() != dev or scales.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    codes, scales = codes.contiguous(), scales.contiguous()
    return (codes, scales), gdn_held(codes.data_ptr(), scales.data_ptr())


def _device(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a GPU device (there is no CPU path)")
    return dev


def _new_checkpoint(x):
    dims = x.shape
    codes = torch.empty_like(x, dtype=torch.int8) if x.is_contiguous() else x.new_empty(dims, dtype=torch.int8)
    groups = (*dims[:-1], -(-dims[-1] // GROUP))
    return Checkpoint(codes, x.new_empty(groups) if x.dtype == torch.bfloat16 else x.new_empty(groups, dtype=torch.bfloat16))


def checkpoint_activation(x):
    """x [..., D] (bf16 or fp32) kept in 8 bits: a Checkpoint, 8.5 bits an element.

    In groups of 32 along the last dimension: a scale (the smallest bfloat16 s with
    127 s >= the group's largest magnitude, 0 below 2^-100) and the integers
    nearest to the elements over it, ties to even.  A group with an infinity or a
    NaN stands for NaNs.  The rows of x may be parts of wider ones.
    """
    dev, code = _gpu(x, "x")
    if x.dim() == 0 or not 0 < x.shape[-1] < 1 << 31:
        raise ValueError("x must be [...,D], 0 < D < 2^31")
    D = x.shape[-1]
    rows = x.reshape(-1, D)
    n = rows.shape[0]
    stride = rows.stride(0) if n > 1 else D
    if (D > 1 and rows.stride(1) != 1) or not D <= stride <= 1 << 31:
        rows, stride = rows.contiguous(), D
    if n >> 31:
        raise ValueError("x must have fewer than 2^31 rows")
    c = _new_checkpoint(x)
    held = gdn_held(c.codes.data_ptr(), c.scales.data_ptr())
    shape = gdn_held_shape(n, D, stride, n, n, code, 8)
    _run(dev, (_lib or _load()).gdn_hold, rows.data_ptr(), None, _addr(held), None, _addr(shape))
    return c


def restore_activation(checkpoint, dtype=torch.bfloat16, out=None):
    """The values that a Checkpoint stands for, rounded once to ``dtype`` (bf16 or
    fp32).  ``out``, a contiguous tensor of the codes' shape, is used as given."""
    codes, scales = checkpoint
    if dtype not in _DTYPES:
        raise ValueError("dtype must be bfloat16 or float32")
    if codes.dim() == 0 or not 0 < codes.shape[-1] < 1 << 31:
        raise ValueError("codes must be [...,D], 0 < D < 2^31")
    dev = _device(codes)
    D = codes.shape[-1]
    n = codes.numel() // D
    if n >> 31:
        raise ValueError("codes must have fewer than 2^31 rows")
    kept, held = _held_rows(checkpoint, n, D, dev, "checkpoint")
    if out is None:
        out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    elif out.shape != codes.shape or out.dtype != dtype or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError(f"out must be a contiguous {dtype} {list(codes.shape)} on cuda:{dev}")
    else:
        _apart("out", [out], *kept)
    shape = gdn_held_shape(n, D, D, n, n, _DTYPES[dtype], 8)
    _run(dev, (_lib or _load()).gdn_restore, _addr(held), None, out.data_ptr(), None, _addr(shape))
    return out


def make_state_cache(state_pool, slots, bits=8):
    """Codes and scales of a cache of ``slots`` slots for the states of
    ``state_pool`` [P, ...], in 8 or 4 bits: (int8 [slots, E], bfloat16
    [slots, ceil(E/32)]) with E elements a state, or uint8 [slots, ceil(E/2)]
    codes."""
    if bits not in (4, 8):
        raise ValueError("bits must be 8 or 4")
    if state_pool.dim() < 2 or state_pool.shape[0] == 0 or state_pool[0].numel() == 0:
        raise ValueError("state_pool must be [P,...] with at least one slot and one element a slot")
    E = state_pool[0].numel()
    codes = state_pool.new_zeros((slots, E if bits == 8 else (E + 1) // 2), dtype=torch.int8 if bits == 8 else torch.uint8)
    return codes, state_pool.new_zeros((slots, -(-E // GROUP)), dtype=torch.bfloat16)


def _cache_args(pool, pool_indices, codes, scales, cache_indices):
    """Checks a cache against a pool; the device, the structs and what they point to."""
    dev, code = _gpu(pool, "state_pool")
    dims = pool.shape
    P = dims[0] if len(dims) > 1 else 0
    if not P or not pool.is_contiguous():
        raise ValueError("state_pool must be a contiguous [P,...]")
    E = pool.numel() // P
    if not 0 < E < 1 << 31 or P >> 31:
        raise ValueError("state_pool must have fewer than 2^31 slots of 1 to 2^31 - 1 elements")
    bits = _CODE_BITS.get(codes.dtype)
    dims = codes.shape
    if bits is None or len(dims) != 2 or dims[1] != (E if bits == 8 else (E + 1) // 2) or not codes.is_contiguous():
        raise ValueError(f"codes must be a contiguous int8 [slots,{E}] (8 bits) or uint8 [slots,{(E + 1) // 2}] (4 bits)")
    C, groups = dims[0], -(-E // GROUP)
    if scales.shape != (C, groups) or scales.dtype != torch.bfloat16 or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous bfloat16 [{C},{groups}]")
    if C >> 31:
        raise ValueError("codes must have fewer than 2^31 slots")
    n, i32 = pool_indices.shape, torch.int32
    if len(n) != 1 or pool_indices.dtype != i32 or cache_indices.dtype != i32 or cache_indices.shape != n:
        raise ValueError("state_indices and cache_indices must be int32 [n], the same n for both")
    if not codes.get_device() == scales.get_device() == pool_indices.get_device() == cache_indices.get_device() == dev:
        raise ValueError(f"codes, scales and the indices must be on cuda:{dev}")
    p, c, s = pool.data_ptr(), codes.data_ptr(), scales.data_ptr()
    p1, c1, s1 = p + P * E * (4 if code else 2), c + C * dims[1], s + 2 * C * groups
    if (p < c1 and c < p1) or (p < s1 and s < p1) or (c < s1 and s < c1):
        raise ValueError("state_pool, codes and scales must not overlap")
    return (dev, gdn_held(c, s), gdn_held_shape(n[0], E, E, P, C, code, bits), pool_indices.contiguous(),
            cache_indices.contiguous(), p)


def state_cache_write(state_pool, state_indices, codes, scales, cache_indices):
    """Writes states into a cache of 8 or 4 bits: slot state_indices[i] of
    state_pool [P, ...] (bf16 or fp32: the delta rule's states, the convolution's
    histories, the linear recurrence's states) goes to slot cache_indices[i] of codes
    and scales (see make_state_cache).  Indices int32 [n]; a pair with an index
    outside its tensor is skipped; no cache slot may be named twice.  The format is
    checkpoint_activation's, in groups of 32 elements of the flattened state; with 4
    bits the integers reach from -7 to 7."""
    dev, held, shape, pi, ci, pool = _cache_args(state_pool, state_indices, codes, scales, cache_indices)
    _run(dev, (_lib or _load()).gdn_hold, pool, pi.data_ptr(), _addr(held), ci.data_ptr(),
         _addr(shape))


def state_cache_read(codes, scales, cache_indices, state_pool, state_indices):
    """Reads states back: slot cache_indices[i] of the cache goes to slot
    state_indices[i] of state_pool, rounded once to its dtype.  Indices as for
    state_cache_write; no pool slot may be named twice."""
    dev, held, shape, pi, ci, pool = _cache_args(state_pool, state_indices, codes, scales, cache_indices)
    _run(dev, (_lib or _load()).gdn_restore, _addr(held), ci.data_ptr(), pool, pi.data_ptr(),
         _addr(shape))


# ---------------------------------------------------------------------------
# The gated RMS norm with its inputs in 8 bits
# ---------------------------------------------------------------------------
def fused_gated_rms_norm_checkpoint(x, z, weight, eps=1e-6, out=None):
    """``fused_gated_rms_norm`` that also keeps x and z in 8 bits for the backward
    pass: ``(y, x_checkpoint, z_checkpoint)``, as checkpoint_activation would give
    them, written in the pass that reads x and z.  y is taken from x and z as they
    are."""
    dev, shape, weight = _norm_args(x, weight)
    z = _gate_rows(x, z, shape)
    x = x.contiguous()
    if out is None:
        out = torch.empty_like(x)
    else:
        _apart("out", [_given(out, x.shape, x, dev, "out")], weight, x, z)
    cx = codes, scales = _new_checkpoint(x)
    cz = Checkpoint(torch.empty_like(codes), torch.empty_like(scales))   # cheaper than new ones by their sizes
    x8, z8 = gdn_held(codes.data_ptr(), scales.data_ptr()), gdn_held(cz.codes.data_ptr(), cz.scales.data_ptr())
    _run(dev, (_lib or _load()).gdn_gated_norm_hold, x.data_ptr(), z.data_ptr(), weight.data_ptr(), eps,
         out.data_ptr(), _addr(x8), _addr(z8), _addr(shape))
    return out, cx, cz


def fused_gated_rms_norm_checkpoint_bwd(x_checkpoint, z_checkpoint, weight, dy, eps=1e-6, workspace=None):
    """Backward pass of ``fused_gated_rms_norm`` at the values that two checkpoints
    stand for: ``(dx, dz, dweight)``, dx and dz in dy's dtype and shape [..., D],
    dweight float32 [D].  ``workspace`` as for fused_gated_rms_norm_bwd."""
    dev, shape, weight = _norm_args(dy, weight)
    dy = dy.contiguous()
    kept_x, x8 = _held_rows(x_checkpoint, shape.rows, shape.D, dev, "x_checkpoint")
    kept_z, z8 = _held_rows(z_checkpoint, shape.rows, shape.D, dev, "z_checkpoint")
    lib = _lib or _load()
    need = _l._load().gdn_norm_bwd_workspace_bytes(_addr(shape))
    ws = _workspace(workspace, need, dev, dy)
    dx, dz = torch.empty_like(dy), torch.empty_like(dy)
    dweight = torch.empty_like(weight, dtype=torch.float32)
    _run(dev, lib.gdn_gated_norm_hold_bwd, _addr(x8), _addr(z8), weight.data_ptr(), eps, dy.data_ptr(), dx.data_ptr(),
         dz.data_ptr(), dweight.data_ptr(), _addr(shape), ws.data_ptr(), need)
    return dx, dz, dweight
