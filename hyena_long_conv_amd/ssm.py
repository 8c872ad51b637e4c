"""The state-space block's operators: residual norm, 8-bit matrix product,
short causal convolution and selective scan, with their single-token and
backward forms.  Python binding of their part of the C ABI in include/hyena.h,
which holds the formulas.

Activations [B, D, L] (or [rows, D] for the norm and the product) are float32
or bfloat16, contiguous and all on one GPU; work is enqueued on the current
stream of that GPU, whichever GPU is the current one.

    a prompt                                        a token
    y, s = rms_norm(x, weight, residual=s)          the same, with one row to a sequence
    q, sc, s = rms_norm_quantized(x, weight, residual=s)
    xz = scaled_matmul(q, sc, wq, wsc, channel_major=True)
    x, cs = short_conv(x, w, b, silu=True,          x = short_conv_step(x, w, cs, b, silu=True)
                       lengths=n, return_state=True)
    y, ss = selective_scan(x, delta, A, Bm, Cm,     y = selective_scan_step(x, delta, A, Bm, Cm, ss, z=z)
                           z=z, lengths=n, return_state=True)
"""
from __future__ import annotations

import ctypes
import os

import hyena_long_conv_amd as _H

i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class ShortConvParams(ctypes.Structure):
    _fields_ = [("B", i64), ("L", i64), ("D", i32), ("T", i32), ("silu", i32), ("reserved", i32),
                ("w", vp), ("bias", vp), ("state", vp), ("lengths", vp)]


class SelectiveScanParams(ctypes.Structure):
    _fields_ = [("B", i64), ("L", i64), ("D", i32), ("G", i32), ("N", i32), ("softplus", i32),
                ("u", vp), ("delta", vp), ("A", vp), ("Bm", vp), ("Cm", vp), ("skip", vp), ("z", vp),
                ("delta_bias", vp), ("state", vp), ("lengths", vp)]


class SelectiveScanGrads(ctypes.Structure):
    _fields_ = [(k, vp) for k in ("gu", "gdelta", "gA", "gB", "gC", "gskip", "gz", "gdelta_bias", "gstate")]


def declare(L):
    """Argument types of the library's functions for this module."""
    cp, sp, gp, f32 = (ctypes.POINTER(ShortConvParams), ctypes.POINTER(SelectiveScanParams),
                       ctypes.POINTER(SelectiveScanGrads), ctypes.c_float)
    for name, args, res in (
            ("hyena_short_conv", [vp, cp, vp, vp, i32, vp], i32),
            ("hyena_short_conv_step", [vp, cp, vp, vp, i32, vp], i32),
            ("hyena_short_conv_backward_workspace_bytes", [i64, i32, i32, i64], i64),
            ("hyena_short_conv_backward", [vp, cp, vp, vp, vp, vp, vp, vp, i32, vp, i64, vp], i32),
            ("hyena_selective_scan_workspace_bytes", [i64, i32, i32, i64], i64),
            ("hyena_selective_scan", [sp, vp, vp, i32, vp, i64, vp], i32),
            ("hyena_selective_scan_step", [sp, vp, vp, i32, vp], i32),
            ("hyena_selective_scan_backward_workspace_bytes", [i64, i32, i32, i32, i64], i64),
            ("hyena_selective_scan_backward", [sp, vp, vp, gp, i32, vp, i64, vp], i32),
            ("hyena_rms_norm", [vp, vp, vp, vp, vp, i64, i32, f32, i32, vp], i32),
            ("hyena_rms_norm_quantized", [vp, vp, vp, vp, vp, vp, i64, i32, f32, i32, vp], i32),
            ("hyena_rms_norm_backward_workspace_bytes", [i64, i32], i64),
            ("hyena_rms_norm_backward", [vp, vp, vp, vp, vp, vp, i64, i32, f32, i32, vp, i64, vp], i32),
            ("hyena_quantize", [vp, vp, vp, i64, i32, i32, i32, vp], i32),
            ("hyena_scaled_matmul", [vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, i32, i32, vp], i32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


# ------------------------------------------------------------------ checking

def _torch():
    import torch
    return torch


def _take(t, name, shape, dtype, device):
    """The address of tensor t, which has to be what the operator takes; None gives 0."""
    if t is None:
        return None
    try:                                              # one expression for a single token's call, where this counts
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _H._need_cuda(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    raise ValueError(f"{name} is on {t.device}, not on {device}")


def _call(name, device, *args):
    """One C-ABI call on the device's current stream, with that device current."""
    import torch
    fn, at = getattr(_H._lib or _H.lib(), name), device.index
    stream = torch._C._cuda_getCurrentRawStream(at)
    if torch._C._cuda_getDevice() == at:
        code = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, stream)
    if code != 0:
        raise _H.HyenaError(code, name)


_POISON = os.environ.get("HYENA_POISON") == "1"       # asked for once: a token's call has no time for it


def _like(t):
    """An output of t's shape and dtype (filled with NaN under the package's test instrument)."""
    import torch
    return _H._empty_like(t) if _POISON else torch.empty_like(t)


def _activation(x, name, dims):
    """Checks the tensor that sets a call's shape, dtype and device: 0 for float32, 1 for bfloat16."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA (ROCm) tensor")
    if x.dim() != dims:
        raise ValueError(f"{name} has {x.dim()} dimensions, not {dims}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _H._io_of(x)


def _dims(t, name, dims):
    """Checks the tensor that sets a call's other sizes."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA (ROCm) tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} has {t.dim()} dimensions, not {dims}")


def _workspace(workspace, nbytes, name, device):
    """(workspace, its address, its bytes): the caller's, or one allocated here."""
    torch = _torch()
    if nbytes < 0:
        raise _H.HyenaError(2, name)
    if workspace is None:
        workspace = _new(nbytes, torch.uint8, device) if nbytes else None
    else:
        _H._need_cuda(workspace, "workspace")
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, not on {device}")
    if workspace is None:
        return None, None, 0
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# --------------------------------------------------------- short convolution

def _conv_params(x, w, bias, silu, state, lengths, B, D, L):
    torch = _torch()
    _dims(w, "w", 2)
    if w.shape[0] != D:
        raise ValueError(f"w shape {tuple(w.shape)} is not [{D}, T]")
    T = w.shape[1]
    dev = x.device
    return T, ShortConvParams(B, L, D, T, int(bool(silu)), 0, _take(w, "w", (D, T), torch.float32, dev),
                              _take(bias, "bias", (D,), torch.float32, dev),
                              _take(state, "state", (B, D, T - 1), x.dtype, dev),
                              _take(lengths, "lengths", (B,), torch.int32, dev))


def short_conv(x, w, bias=None, silu: bool = False, state=None, lengths=None, return_state: bool = False, out=None,
               state_out=None):
    """y[t] = act(bias + sum_j w[:, j] x[t-j]) of x [B, D, L] with w [D, T] and
    bias [D] in float32; silu: act(p) = p * sigmoid(p).  state [B, D, T-1]
    holds the inputs before x, oldest first.  lengths (int32 [B]): steps of
    each sequence; y is zero behind them.  Returns y, with return_state (y,
    the last T-1 inputs [B, D, T-1])."""
    io = _activation(x, "x", 3)
    B, D, L = x.shape
    T, p = _conv_params(x, w, bias, silu, state, lengths, B, D, L)
    y = _like(x) if out is None else out
    yp = y.data_ptr() if out is None else _take(out, "out", x.shape, x.dtype, x.device)
    if return_state and state_out is None:
        state_out = _new((B, D, T - 1), x.dtype, x.device)
    so = _take(state_out, "state_out", (B, D, T - 1), x.dtype, x.device) if T > 1 else None
    _call("hyena_short_conv", x.device, x.data_ptr(), ctypes.byref(p), yp, so, io)
    return (y, state_out) if return_state else y


def short_conv_step(x, w, state, bias=None, silu: bool = False, out=None):
    """One token for each sequence: x [B, D] -> y [B, D]; state [B, D, T-1]
    (None with T = 1) moves on by one in place."""
    io = _activation(x, "x", 2)
    B, D = x.shape
    T, p = _conv_params(x, w, bias, silu, None, None, B, D, 1)
    dev, t = x.device, x.dtype
    y = _like(x) if out is None else out
    yp = y.data_ptr() if out is None else _take(out, "out", (B, D), t, dev)
    st = _take(state, "state", (B, D, T - 1), t, dev) if T > 1 else None
    _call("hyena_short_conv_step", dev, x.data_ptr(), ctypes.byref(p), st, yp, io)
    return y


def short_conv_backward_workspace_bytes(B: int, D: int, T: int, L: int) -> int:
    return int(_H.lib().hyena_short_conv_backward_workspace_bytes(B, D, T, L))


def short_conv_backward(x, w, gy, bias=None, silu: bool = False, state=None, lengths=None, gstate_out=None,
                        workspace=None):
    """Gradients (gx, gw, gbias, gstate) of a loss with dloss/dy = gy through
    short_conv of the same arguments; gstate_out is the loss's gradient with
    respect to the returned state.  gbias is None without a bias, gstate
    without a state."""
    torch = _torch()
    io = _activation(x, "x", 3)
    B, D, L = x.shape
    T, p = _conv_params(x, w, bias, silu, state, lengths, B, D, L)
    dev = x.device
    gx, gw = _like(x), _like(w)
    gbias = _like(bias) if bias is not None else None
    gstate = _like(state) if state is not None else None
    gso = _take(gstate_out, "gstate_out", (B, D, T - 1), x.dtype, dev) if T > 1 else None
    keep, ws, wsb = _workspace(workspace, short_conv_backward_workspace_bytes(B, D, T, L),
                               "hyena_short_conv_backward_workspace_bytes", dev)
    _call("hyena_short_conv_backward", dev, x.data_ptr(), ctypes.byref(p), _take(gy, "gy", x.shape, x.dtype, dev), gso,
          gx.data_ptr(), gw.data_ptr(), _take(gbias, "gbias", (D,), torch.float32, dev),
          gstate.data_ptr() if gstate is not None and T > 1 else None, io, ws, wsb)
    return gx, gw, gbias, gstate


# ------------------------------------------------------------ selective scan

def _scan_params(u, delta, A, Bm, Cm, skip, z, delta_bias, softplus, state, lengths, B, D, tail):
    torch = _torch()
    dev, t, f32 = u.device, u.dtype, torch.float32
    _dims(A, "A", 2)
    if A.shape[0] != D:
        raise ValueError(f"A shape {tuple(A.shape)} is not [{D}, N]")
    N = A.shape[1]
    _dims(Bm, "Bm", 3 + len(tail))
    G = Bm.shape[1]
    bc = (B, G, N, *tail)
    return N, G, SelectiveScanParams(
        B, tail[0] if tail else 1, D, G, N, int(bool(softplus)), u.data_ptr(),
        _take(delta, "delta", u.shape, t, dev), _take(A, "A", (D, N), f32, dev), _take(Bm, "Bm", bc, t, dev),
        _take(Cm, "Cm", bc, t, dev), _take(skip, "skip", (D,), f32, dev), _take(z, "z", u.shape, t, dev),
        _take(delta_bias, "delta_bias", (D,), f32, dev), _take(state, "state", (B, D, N), f32, dev),
        _take(lengths, "lengths", (B,), torch.int32, dev))


def selective_scan_workspace_bytes(B: int, D: int, N: int, L: int) -> int:
    return int(_H.lib().hyena_selective_scan_workspace_bytes(B, D, N, L))


def selective_scan(u, delta, A, Bm, Cm, skip=None, z=None, delta_bias=None, softplus: bool = True, state=None,
                   lengths=None, return_state: bool = False, out=None, state_out=None, workspace=None):
    """y [B, D, L] of the scan h[t] = exp(dt[t] A) h[t-1] + dt[t] u[t] Bm[t],
    y[t] = (sum_n Cm[t] h[t] + skip u[t]) * z[t] sigmoid(z[t]), with dt =
    softplus(delta + delta_bias) (softplus=False: the sum itself).  u, delta,
    z [B, D, L]; Bm, Cm [B, G, N, L], each for D/G channels; A [D, N], skip
    and delta_bias [D], state [B, D, N] in float32; lengths int32 [B].
    Returns y, with return_state (y, h at each sequence's end [B, D, N])."""
    torch = _torch()
    io = _activation(u, "u", 3)
    B, D, L = u.shape
    N, G, p = _scan_params(u, delta, A, Bm, Cm, skip, z, delta_bias, softplus, state, lengths, B, D, (L,))
    dev = u.device
    y = _like(u) if out is None else out
    yp = y.data_ptr() if out is None else _take(out, "out", u.shape, u.dtype, dev)
    if return_state and state_out is None:
        state_out = _new((B, D, N), torch.float32, dev)
    keep, ws, wsb = _workspace(workspace, selective_scan_workspace_bytes(B, D, N, L),
                               "hyena_selective_scan_workspace_bytes", dev)
    _call("hyena_selective_scan", dev, ctypes.byref(p), yp,
          _take(state_out, "state_out", (B, D, N), torch.float32, dev), io, ws, wsb)
    return (y, state_out) if return_state else y


def selective_scan_step(u, delta, A, Bm, Cm, state, skip=None, z=None, delta_bias=None, softplus: bool = True,
                        out=None):
    """One token for each sequence: u, delta, z [B, D], Bm, Cm [B, G, N] -> y
    [B, D]; state [B, D, N] float32 moves on by one in place."""
    torch = _torch()
    io = _activation(u, "u", 2)
    B, D = u.shape
    N, G, p = _scan_params(u, delta, A, Bm, Cm, skip, z, delta_bias, softplus, None, None, B, D, ())
    dev = u.device
    y = _like(u) if out is None else out
    yp = y.data_ptr() if out is None else _take(out, "out", (B, D), u.dtype, dev)
    _call("hyena_selective_scan_step", dev, ctypes.byref(p), _take(state, "state", (B, D, N), torch.float32, dev), yp,
          io)
    return y


def selective_scan_backward_workspace_bytes(B: int, D: int, G: int, N: int, L: int) -> int:
    return int(_H.lib().hyena_selective_scan_backward_workspace_bytes(B, D, G, N, L))


def selective_scan_backward(u, delta, A, Bm, Cm, gy, skip=None, z=None, delta_bias=None, softplus: bool = True,
                            state=None, lengths=None, gstate_out=None, workspace=None) -> dict:
    """Gradients of a loss with dloss/dy = gy (and dloss/dh = gstate_out at the
    sequences' ends) through selective_scan of the same arguments: a dict of
    gu, gdelta, gA, gB, gC, gskip, gz, gdelta_bias and gstate, None where the
    argument is None."""
    torch = _torch()
    io = _activation(u, "u", 3)
    B, D, L = u.shape
    N, G, p = _scan_params(u, delta, A, Bm, Cm, skip, z, delta_bias, softplus, state, lengths, B, D, (L,))
    dev = u.device
    out = dict(gu=u, gdelta=delta, gA=A, gB=Bm, gC=Cm, gskip=skip, gz=z, gdelta_bias=delta_bias, gstate=state)
    out = {k: _like(v) if v is not None else None for k, v in out.items()}
    g = SelectiveScanGrads(*[v.data_ptr() if v is not None else None for v in out.values()])
    keep, ws, wsb = _workspace(workspace, selective_scan_backward_workspace_bytes(B, D, G, N, L),
                               "hyena_selective_scan_backward_workspace_bytes", dev)
    _call("hyena_selective_scan_backward", dev, ctypes.byref(p), _take(gy, "gy", u.shape, u.dtype, dev),
          _take(gstate_out, "gstate_out", (B, D, N), torch.float32, dev), ctypes.byref(g), io, ws, wsb)
    return out


# -------------------------------------------------------------- residual norm

def _rows(x, name):
    _H._need_cuda(x, name)
    io = _H._io_of(x)
    if x.dim() < 1:
        raise ValueError(f"{name} has no dimension")
    D = x.shape[-1]
    return io, x.numel() // D if D else 0, D


def rms_norm(x, weight, residual=None, eps: float = 1e-6, out=None):
    """s / sqrt(mean(s^2) + eps) * weight along the last axis, with s = x +
    residual.  Returns y, with a residual (y, s), s as stored in x's dtype."""
    torch = _torch()
    io, rows, D = _rows(x, "x")
    dev = x.device
    y = _like(x) if out is None else out
    yp = y.data_ptr() if out is None else _take(out, "out", x.shape, x.dtype, dev)
    s = _like(x) if residual is not None else None
    _call("hyena_rms_norm", dev, x.data_ptr(), _take(residual, "residual", x.shape, x.dtype, dev),
          _take(weight, "weight", (D,), torch.float32, dev), yp, s.data_ptr() if s is not None else None, rows, D, eps,
          io)
    return (y, s) if residual is not None else y


def _new(shape, dtype, dev):
    """An output, filled with NaN under the package's test instrument."""
    import torch
    t = torch.empty(shape, dtype=dtype, device=dev)
    if _POISON:
        _H._poison(t if dtype.itemsize > 1 else t.view(torch.uint8))
    return t


def _codes(shape, dev, block_rows=1):
    """Codes and scales for values [..., K]: a scale for each 128 of a row, or for each 128 x 128."""
    import torch
    head = shape[:-1] if block_rows == 1 else (-(-shape[0] // 128),)
    return (_new(shape, torch.float8_e4m3fn, dev), _new((*head, -(-shape[-1] // 128)), torch.float32, dev))


def rms_norm_quantized(x, weight, residual=None, eps: float = 1e-6):
    """rms_norm with its output in 8 bits: (q, scales) or, with a residual,
    (q, scales, s); q float8_e4m3fn of x's shape, scales float32 [...,
    ceil(D/128)], one for each 128 values of a row."""
    torch = _torch()
    io, rows, D = _rows(x, "x")
    dev = x.device
    q, scales = _codes(x.shape, dev)
    s = _like(x) if residual is not None else None
    _call("hyena_rms_norm_quantized", dev, x.data_ptr(), _take(residual, "residual", x.shape, x.dtype, dev),
          _take(weight, "weight", (D,), torch.float32, dev), q.data_ptr(), scales.data_ptr(),
          s.data_ptr() if s is not None else None, rows, D, eps, io)
    return (q, scales, s) if residual is not None else (q, scales)


def rms_norm_backward_workspace_bytes(rows: int, D: int) -> int:
    return int(_H.lib().hyena_rms_norm_backward_workspace_bytes(rows, D))


def rms_norm_backward(s, weight, gy, gs=None, eps: float = 1e-6, workspace=None):
    """(gx, gweight) of a loss with dloss/dy = gy through rms_norm, from the
    normed sum s; gs, the gradient that reaches s past the norm, is added to
    gx, which is the gradient of x and of residual alike."""
    torch = _torch()
    io, rows, D = _rows(s, "s")
    dev = s.device
    gx, gw = _like(s), _new((D,), torch.float32, dev)
    keep, ws, wsb = _workspace(workspace, rms_norm_backward_workspace_bytes(rows, D),
                               "hyena_rms_norm_backward_workspace_bytes", dev)
    _call("hyena_rms_norm_backward", dev, s.data_ptr(), _take(weight, "weight", (D,), torch.float32, dev),
          _take(gy, "gy", s.shape, s.dtype, dev), _take(gs, "gs", s.shape, s.dtype, dev), gx.data_ptr(), gw.data_ptr(),
          rows, D, eps, io, ws, wsb)
    return gx, gw


# -------------------------------------------------------------- 8-bit product

def quantize(x, block_rows: int = 1):
    """(q, scales) of x [..., K]: float8_e4m3fn codes with a float32 scale for
    each 128 values of a row (block_rows=1, scales [..., ceil(K/128)]) or, for
    a weight [N, K], for each 128 x 128 values (block_rows=128)."""
    io, rows, K = _rows(x, "x")
    if block_rows != 1 and x.dim() != 2:
        raise ValueError("blocks of several rows are for matrices")
    q, scales = _codes(x.shape, x.device, block_rows)
    _call("hyena_quantize", x.device, x.data_ptr(), q.data_ptr(), scales.data_ptr(), rows, K, block_rows, io)
    return q, scales


def scaled_matmul(q, scales, wq, wscales, bias=None, out_dtype=None, channel_major: bool = False, out=None):
    """The product of values given as codes and scales (quantize,
    rms_norm_quantized): left [..., K] times right [N, K] transposed, plus bias
    [N] (float32), in out_dtype (bfloat16 by default, or float32).  Returns
    [..., N], with channel_major [N, M] of a left [M, K], or [B, N, L] of a
    left [B, L, K], the layout of the convolutions and the scan.  Sums are fp32;
    for bfloat16 outputs of more than 64 rows those of 8 neighbouring products
    lose what is below 2^-13 of the largest one."""
    torch = _torch()
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    _H._need_cuda(q, "q", e4m3)
    dev = q.device
    _dims(wq, "wq", 2)
    if q.dim() < 2 or q.shape[-1] != wq.shape[1]:
        raise ValueError(f"shapes {tuple(q.shape)} and {tuple(wq.shape)} do not make a product")
    if channel_major and q.dim() > 3:
        raise ValueError("channel_major takes [M, K] or [B, L, K]")
    N, K = wq.shape
    kb = -(-K // 128)
    L = q.shape[-2]
    B = q.numel() // (L * K) if L * K else 0
    out_dtype = out_dtype or (out.dtype if out is not None else torch.bfloat16)
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be float32 or bfloat16")
    shape = (*q.shape[:-2], N, L) if channel_major else (*q.shape[:-1], N)
    o = _new(shape, out_dtype, dev) if out is None else out
    op = o.data_ptr() if out is None else _take(out, "out", shape, out_dtype, dev)
    _call("hyena_scaled_matmul", dev, q.data_ptr(), _take(scales, "scales", (*q.shape[:-1], kb), f32, dev),
          _take(wq, "wq", (N, K), e4m3, dev), _take(wscales, "wscales", (-(-N // 128), kb), f32, dev),
          _take(bias, "bias", (N,), f32, dev), op, B, L, N, K, int(bool(channel_major)),
          _H.HYENA_FP32 if out_dtype == f32 else _H.HYENA_BF16)
    return o
