"""Mixer operators of libkda.so: the short causal convolution, the selective
scan and the group norm with its gate (the "mixer operators" of include/kda.h).

Argument marshalling only, as in ``kda.py``: every step runs in the HIP
kernels, torch supplies device memory and the current stream.  Token tensors
are bf16 or fp32; parameters, their gradients and scan states are fp32.

A call has sequences of one length ([B, T, ...] tensors) or, with
``cu_seqlens`` (int32 [N + 1] on the same device), a packed batch
([T_total, ...] tensors).  Inputs may be slices of wider projections: the
trailing dimensions must be contiguous and the token rows evenly spaced.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import kda as _k
from .kda import KDA_OK, KDAError, _dtype_code

_INT_MAX = 2 ** 31 - 1
_ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _device(x: torch.Tensor) -> int:
    """The GPU's index.  (The checks compare indices and let torch make outputs
    like their inputs: on one-token calls the host's steps are what counts.)"""
    if not x.is_cuda:
        raise ValueError("the mixer operators run on the GPU, got a tensor on %s" % x.device)
    return x.get_device()


def _like(x: torch.Tensor) -> torch.Tensor:
    """A new contiguous tensor of x's shape and dtype."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _f32(dev: int, *shape) -> torch.Tensor:
    return torch.empty(shape, dtype=torch.float32, device=dev)


def _act(name) -> int:
    try:
        return _ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError("activation is None, 'silu' or 'sigmoid', got %r" % (name,)) from None


def _call(name: str, dev: int, *args):
    """The C call on GPU dev and its current stream."""
    fn = getattr(_k.load_library(), name)
    # the raw handle: a Stream object would cost as much as a small launch
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    else:
        st = fn(*args, stream)
    if st != KDA_OK:
        raise KDAError(st, name)


def _size(name: str, *args) -> int:
    """The bytes of a workspace; 0 for sizes that are refused: the call, which
    checks them first, then says why."""
    n = getattr(_k.load_library(), name)(*args)
    return 0 if n == ctypes.c_size_t(-1).value else int(n)


def _workspace(workspace: Optional[torch.Tensor], need: int, dev: int):
    """The caller's workspace if it is large enough, else a new one; and its bytes."""
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous on cuda:%d" % dev)
        have = workspace.numel() * workspace.element_size()
        if have >= need:
            return workspace, have
    if need == 0:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=dev), need


def _refuse(t: torch.Tensor, name: str, shape, dtype, dev: int):
    """What is wrong with a tensor, in the order the checks name it."""
    if t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d" % (name, dev))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))


def _check(t: torch.Tensor, name: str, shape, dtype, dev: int):
    if t.shape == shape and t.dtype == dtype and t.is_contiguous() and t.get_device() == dev:
        return
    _refuse(t, name, shape, dtype, dev)
    raise ValueError("%s must be contiguous" % name)


def _fits(shape, lead: int, name: str):
    """Refuses sizes that the C calls' ints do not hold."""
    tokens = 1
    for n in shape[:lead]:
        tokens *= n
    if tokens > _INT_MAX or max(shape) > _INT_MAX:
        raise KDAError(_k.KDA_ERR_UNSUPPORTED, "%s of %d rows" % (name, tokens))


def _rows(t: torch.Tensor, name: str, shape, lead: int, dtype, dev: int) -> int:
    """Checks a token tensor whose first `lead` dimensions count tokens;
    returns the elements between its token rows."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        _refuse(t, name, shape, dtype, dev)
    if t.numel() > _INT_MAX:
        _fits(shape, lead, name)
    width = 1
    for n in shape[lead:]:
        width *= n
    if t.is_contiguous():
        return width
    stride = t.stride()
    inner = 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] != 1 and stride[d] != inner:
            raise ValueError("%s must be contiguous in its last %d dimensions" % (name, len(shape) - lead))
        inner *= shape[d]
    row, span = None, 0     # token stride, and the stride the next outer dimension must have
    for d in range(lead - 1, -1, -1):
        if shape[d] == 1:
            continue
        if row is None:
            row, span = stride[d], stride[d] * shape[d]
            if row < width:     # one row for all tokens (an expanded tensor), or rows that overlap
                raise ValueError("%s must have token rows of its own" % name)
        elif stride[d] != span:
            raise ValueError("%s must have evenly spaced token rows" % name)
        else:
            span *= shape[d]
    return width if row is None else row


def _seqs(x: torch.Tensor, cu_seqlens: Optional[torch.Tensor], lead: int):
    """(N, T) of a call: N sequences of T tokens, or of a packed axis of T."""
    if cu_seqlens is None:
        if x.dim() < lead + 1:
            raise ValueError("x has too few dimensions")
        return x.shape[0], x.shape[1]
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32 [N + 1]")
    if cu_seqlens.get_device() != x.get_device() or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous on %s" % x.device)
    return cu_seqlens.numel() - 1, x.shape[0]


# ---- short convolution ----------------------------------------------------------------
def _conv_args(x, weight, bias, state, cu_seqlens):
    dev = _device(x)
    lead = 2 if cu_seqlens is None else 1
    if x.dim() != lead + 1:
        raise ValueError("x is [B, T, D], or [T_total, D] with cu_seqlens")
    N, T = _seqs(x, cu_seqlens, lead)
    D = x.shape[-1]
    if weight.dim() != 2:
        raise ValueError("weight is [D, W]")
    W = weight.shape[1]
    stride = _rows(x, "x", x.shape, lead, x.dtype, dev)
    _check(weight, "weight", (D, W), torch.float32, dev)
    if bias is not None:
        _check(bias, "bias", (D,), torch.float32, dev)
    if state is not None:
        _check(state, "initial_state", (N, W - 1, D), x.dtype, dev)
    return dev, N, T, D, W, _dtype_code(x.dtype), stride


def short_conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True, *,
                   activation="silu", cu_seqlens: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None):
    """Short causal depthwise convolution through ``kda_short_conv_fwd``.

    x: [B, T, D], or packed [T_total, D]; weight: [D, W] fp32, W 2 to 4; bias:
    [D] fp32 or None; initial_state: [N, W - 1, D] in x's dtype, the rows
    before each sequence, or None (zeros); activation: None, "silu" or
    "sigmoid".  Returns (y like x, final_state [N, W - 1, D] or None).  Rows of
    a packed ``out`` behind the last sequence are left as they are.
    """
    dev, N, T, D, W, code, stride = _conv_args(x, weight, bias, initial_state, cu_seqlens)
    act = _act(activation)
    if out is None:
        out = _like(x)
    else:
        _check(out, "out", x.shape, x.dtype, dev)
    if final_state is not None:
        _check(final_state, "final_state", (N, W - 1, D), x.dtype, dev)
    elif output_final_state:
        final_state = torch.empty((N, W - 1, D), dtype=x.dtype, device=dev)
    _call("kda_short_conv_fwd", dev, N, _p(cu_seqlens), T, D, W, code, act, _p(x), stride, _p(weight), _p(bias),
          _p(initial_state), _p(out), _p(final_state))
    return out, final_state


def short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], d_y: torch.Tensor,
                   initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None, *,
                   activation="silu", cu_seqlens: Optional[torch.Tensor] = None,
                   want_d_initial_state: Optional[bool] = None, dx: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of ``short_conv_fwd`` through ``kda_short_conv_bwd``: (dx,
    dweight [D, W], dbias [D] or None, d_initial_state or None).  dbias comes
    with a bias, d_initial_state with an initial_state unless
    ``want_d_initial_state`` says otherwise."""
    dev, N, T, D, W, code, stride = _conv_args(x, weight, bias, initial_state, cu_seqlens)
    act = _act(activation)
    _check(d_y, "d_y", x.shape, x.dtype, dev)
    if d_final_state is not None:
        _check(d_final_state, "d_final_state", (N, W - 1, D), x.dtype, dev)
    if dx is None:
        dx = _like(x)
    else:
        _check(dx, "dx", x.shape, x.dtype, dev)
    dw = _f32(dev, D, W)
    db = _f32(dev, D) if bias is not None else None
    if want_d_initial_state is None:
        want_d_initial_state = initial_state is not None
    ds = torch.empty((N, W - 1, D), dtype=x.dtype, device=dev) if want_d_initial_state else None
    need = _size("kda_short_conv_bwd_workspace_size", N, int(cu_seqlens is not None), T, D, W, code)
    workspace, have = _workspace(workspace, need, dev)
    _call("kda_short_conv_bwd", dev, N, _p(cu_seqlens), T, D, W, code, act, _p(x), stride, _p(weight), _p(bias),
          _p(initial_state), _p(d_y), _p(d_final_state), _p(dx), _p(dw), _p(db), _p(ds), _p(workspace), have)
    return dx, dw, db, ds


def short_conv_step(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], state: torch.Tensor, *,
                    activation="silu", out: Optional[torch.Tensor] = None):
    """One token of N sequences through ``kda_short_conv_step``: x [N, D],
    state [N, W - 1, D] updated in place.  Returns y [N, D]."""
    dev = _device(x)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x is [N, D] and weight [D, W]")
    N, D = x.shape
    W = weight.shape[1]
    act = _act(activation)
    stride = _rows(x, "x", x.shape, 1, x.dtype, dev)
    _check(weight, "weight", (D, W), torch.float32, dev)
    if bias is not None:
        _check(bias, "bias", (D,), torch.float32, dev)
    _check(state, "state", (N, W - 1, D), x.dtype, dev)
    if out is None:
        out = _like(x)
    else:
        _check(out, "out", (N, D), x.dtype, dev)
    _call("kda_short_conv_step", dev, N, D, W, _dtype_code(x.dtype), act, _p(x), stride, _p(weight), _p(bias),
          _p(state), _p(out))
    return out


# ---- selective scan ---------------------------------------------------------------------
def _scan_args(x, dt, A, B, C, D, dt_bias, lead):
    dev = _device(x)
    if x.dim() != lead + 2 or B.dim() != lead + 2:
        raise ValueError("x is [%s, H, P] and B [%s, G, K]" % (("B, T",) * 2 if lead == 2 else ("tokens",) * 2))
    H, P = x.shape[-2:]
    G, K = B.shape[-2:]
    head = x.shape[:lead]
    ty = x.dtype
    code = _dtype_code(ty)
    xs = _rows(x, "x", x.shape, lead, ty, dev)
    bs = _rows(B, "B", head + (G, K), lead, ty, dev)
    cs = _rows(C, "C", head + (G, K), lead, ty, dev)
    ds = _rows(dt, "dt", head + (H,), lead, ty, dev)
    _check(A, "A", (H,), torch.float32, dev)
    if D is not None:
        _check(D, "D", (H,), torch.float32, dev)
    if dt_bias is not None:
        _check(dt_bias, "dt_bias", (H,), torch.float32, dev)
    return dev, H, G, K, P, code, xs, ds, bs, cs


def selective_scan_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                       D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                       initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True, *,
                       dt_softplus: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Selective scan of prompts through ``kda_selective_scan_fwd``:

        S_t = exp(delta_t A) S_{t-1} + delta_t B_t x_t^T,  y_t = S_t^T C_t + D x_t

    with delta = softplus(dt + dt_bias) (``dt_softplus``) or dt + dt_bias.
    x: [B, T, H, P]; dt: [B, T, H]; B, C: [B, T, G, K] (G divides H); packed:
    the same without the batch dimension.  A, D, dt_bias: [H] fp32; states
    [N, H, K, P] fp32.  Returns (y like x, final_state or None);
    ``final_state`` may be ``initial_state`` itself.  The work is done in chunks
    of 64 tokens: a NaN or infinity reaches its own sequence from the start of its
    chunk on (the recurrence and the one-token step: from its token on), never
    another sequence.
    """
    lead = 2 if cu_seqlens is None else 1
    dev, H, G, K, P, code, xs, ds, bs, cs = _scan_args(x, dt, A, B, C, D, dt_bias, lead)
    N, T = _seqs(x, cu_seqlens, lead)
    if initial_state is not None:
        _check(initial_state, "initial_state", (N, H, K, P), torch.float32, dev)
    if out is None:
        out = _like(x)
    else:
        _check(out, "out", x.shape, x.dtype, dev)
    if final_state is not None:
        _check(final_state, "final_state", (N, H, K, P), torch.float32, dev)
    elif output_final_state:
        final_state = _f32(dev, N, H, K, P)
    need = _size("kda_selective_scan_fwd_workspace_size", N, int(cu_seqlens is not None), T, H, G, K, P, code)
    workspace, have = _workspace(workspace, need, dev)
    _call("kda_selective_scan_fwd", dev, N, _p(cu_seqlens), T, H, G, K, P, code, int(bool(dt_softplus)), _p(x), xs,
          _p(dt), ds, _p(A), _p(B), bs, _p(C), cs, _p(D), _p(dt_bias), _p(initial_state), _p(out), _p(final_state),
          _p(workspace), have)
    return out, final_state


def _out_rows(t, name, shape, lead, dtype, dev):
    """An output that may be a view of a wider buffer, or a new tensor; and its row stride."""
    if t is None:
        width = 1
        for n in shape[lead:]:
            width *= n
        return torch.empty(shape, dtype=dtype, device=dev), width
    return t, _rows(t, name, shape, lead, dtype, dev)


def selective_scan_bwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                       D: Optional[torch.Tensor], dt_bias: Optional[torch.Tensor], d_y: torch.Tensor,
                       initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None, *,
                       dt_softplus: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
                       want_d_initial_state: Optional[bool] = None, dx: Optional[torch.Tensor] = None,
                       dB: Optional[torch.Tensor] = None, dC: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Gradients of ``selective_scan_fwd`` through ``kda_selective_scan_bwd``:
    (dx, ddt, dA, dB, dC, dD, ddt_bias, d_initial_state), None where the
    forward has no such input (d_initial_state: unless
    ``want_d_initial_state`` says otherwise).  ``dx``, ``dB`` and ``dC`` may be
    passed as views of one wider buffer."""
    lead = 2 if cu_seqlens is None else 1
    dev, H, G, K, P, code, xs, ds, bs, cs = _scan_args(x, dt, A, B, C, D, dt_bias, lead)
    N, T = _seqs(x, cu_seqlens, lead)
    ty = x.dtype
    _check(d_y, "d_y", x.shape, ty, dev)
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            _check(t, name, (N, H, K, P), torch.float32, dev)
    dx, dxs = _out_rows(dx, "dx", x.shape, lead, ty, dev)
    dB, dbs = _out_rows(dB, "dB", B.shape, lead, ty, dev)
    dC, dcs = _out_rows(dC, "dC", B.shape, lead, ty, dev)
    ddt = torch.empty(x.shape[:-1], dtype=ty, device=dev)
    dA = _f32(dev, H)
    dD = _f32(dev, H) if D is not None else None
    dbias = _f32(dev, H) if dt_bias is not None else None
    if want_d_initial_state is None:
        want_d_initial_state = initial_state is not None
    ds0 = _f32(dev, N, H, K, P) if want_d_initial_state else None
    need = _size("kda_selective_scan_bwd_workspace_size", N, int(cu_seqlens is not None), T, H, G, K, P, code)
    workspace, have = _workspace(workspace, need, dev)
    _call("kda_selective_scan_bwd", dev, N, _p(cu_seqlens), T, H, G, K, P, code, int(bool(dt_softplus)), _p(x), xs,
          _p(dt), ds, _p(A), _p(B), bs, _p(C), cs, _p(D), _p(dt_bias), _p(initial_state), _p(d_y),
          _p(d_final_state), _p(dx), dxs, _p(ddt), _p(dA), _p(dB), dbs, _p(dC), dcs, _p(dD), _p(dbias), _p(ds0),
          _p(workspace), have)
    return dx, ddt, dA, dB, dC, dD, dbias, ds0


def selective_scan_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        D: Optional[torch.Tensor], dt_bias: Optional[torch.Tensor], state: torch.Tensor, *,
                        dt_softplus: bool = False, out: Optional[torch.Tensor] = None):
    """One token of N sequences through ``kda_selective_scan_step``: x [N, H, P],
    dt [N, H], B, C [N, G, K]; state [N, H, K, P] fp32 is updated in place.
    Returns y [N, H, P]."""
    dev, H, G, K, P, code, xs, ds, bs, cs = _scan_args(x, dt, A, B, C, D, dt_bias, 1)
    N = x.shape[0]
    _check(state, "state", (N, H, K, P), torch.float32, dev)
    if out is None:
        out = _like(x)
    else:
        _check(out, "out", x.shape, x.dtype, dev)
    _call("kda_selective_scan_step", dev, N, H, G, K, P, code, int(bool(dt_softplus)), _p(x), xs, _p(dt), ds, _p(A),
          _p(B), bs, _p(C), cs, _p(D), _p(dt_bias), _p(state), _p(out))
    return out


# ---- group norm -------------------------------------------------------------------------
def _norm_args(x, groups, weight, bias, gate):
    dev = _device(x)
    if x.dim() < 1:
        raise ValueError("x is [..., C]")
    C = x.shape[-1]
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    lead = x.dim() - 1
    xs = _rows(x, "x", x.shape, lead, x.dtype, dev)
    zs = _rows(gate, "gate", x.shape, lead, x.dtype, dev) if gate is not None else C
    if weight is not None:
        _check(weight, "weight", (C,), torch.float32, dev)
    if bias is not None:
        _check(bias, "bias", (C,), torch.float32, dev)
    return dev, rows, C, _dtype_code(x.dtype), xs, zs


def group_norm_fwd(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, *,
                   activation="silu", gate_first: bool = False, center: bool = False, eps: float = 1e-5,
                   out: Optional[torch.Tensor] = None):
    """Group norm of the last dimension's ``groups`` groups, each token by
    itself, through ``kda_group_norm_fwd``: act(n) without a gate (a plain norm
    is ``activation=None``), n act(gate) with one, or n of x act(gate) with
    ``gate_first``.  ``center`` subtracts
    the group's mean (else root mean square).  x, gate: [..., C]; weight,
    bias: [C] fp32 or None.  ``out`` may be x or gate itself."""
    dev, rows, C, code, xs, zs = _norm_args(x, groups, weight, bias, gate)
    act = _act(activation)
    if out is None:
        out = _like(x)
    else:
        _check(out, "out", x.shape, x.dtype, dev)
    _call("kda_group_norm_fwd", dev, rows, C, int(groups), code, act, int(bool(center)), int(bool(gate_first)),
          float(eps), _p(x), xs, _p(weight), _p(bias), _p(gate), zs, _p(out))
    return out


def group_norm_bwd(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                   gate: Optional[torch.Tensor], d_y: torch.Tensor, *, activation="silu", gate_first: bool = False,
                   center: bool = False, eps: float = 1e-5, workspace: Optional[torch.Tensor] = None):
    """Gradients of ``group_norm_fwd`` through ``kda_group_norm_bwd``: (dx,
    dweight [C] or None, dbias [C] or None, dgate or None), each where the
    forward has the input."""
    dev, rows, C, code, xs, zs = _norm_args(x, groups, weight, bias, gate)
    act = _act(activation)
    _check(d_y, "d_y", x.shape, x.dtype, dev)
    dx = _like(x)
    dz = _like(x) if gate is not None else None
    dw = _f32(dev, C) if weight is not None else None
    db = _f32(dev, C) if bias is not None else None
    need = 0
    if dw is not None or db is not None:
        need = _size("kda_group_norm_bwd_workspace_size", rows, C, int(groups), code)
    workspace, have = _workspace(workspace, need, dev)
    _call("kda_group_norm_bwd", dev, rows, C, int(groups), code, act, int(bool(center)), int(bool(gate_first)),
          float(eps), _p(x), xs, _p(weight), _p(bias), _p(gate), zs, _p(d_y), _p(dx), _p(dw), _p(db), _p(dz),
          _p(workspace), have)
    return dx, dw, db, dz
