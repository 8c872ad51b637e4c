"""The linear-attention block's operators: rotary positions, linear attention
with a decay for each head, and the norm of each head's outputs with a gate,
with their single-token and backward forms.  Python binding of their part of
the C ABI in include/hyena.h, which holds the formulas.

Activations are token-major, [B, L, heads, head size] (a token: [B, heads, head
size]), float32 or bfloat16 and all on one GPU; work is enqueued on the current
stream of that GPU, whichever GPU is the current one.  q, k, v and what rotary
reads may be parts of wider rows (a head's values are contiguous, the other
strides are free); everything else is contiguous.

    a prompt                                          a token
    freq, f = rotary_frequencies(64)
    rotary(qk, freq, scale=f, out=qk)                 rotary(qk, freq, positions, scale=f, out=qk)
    o, s = linear_attention(q, k, v, log_decay,       o = linear_attention_step(q, k, v, s, log_decay)
                            lengths=n, return_state=True)
    y = group_norm(o.flatten(2), heads, w, b, z=z)    y = group_norm(o.flatten(1), heads, w, b, z=z)
"""
from __future__ import annotations

import ctypes
import math

import hyena_long_conv_amd as _H

from .ssm import _call, _like, _new, _rows, _take, _torch, _workspace

i32, i64, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


def _stride3(name):
    """The members of an int64_t[3], each a field of its own: plain numbers are quicker to hand over than an array."""
    return [(f"{name}_{of}", i64) for of in ("sequence", "token", "head")]


class LinearAttentionParams(ctypes.Structure):
    _fields_ = [("B", i64), ("L", i64), ("H", i32), ("Hq", i32), ("Hk", i32), ("Hv", i32), ("Dk", i32), ("Dv", i32),
                ("scale", f32), ("reserved", i32), ("q", vp), ("k", vp), ("v", vp), *_stride3("q_stride"),
                *_stride3("k_stride"), *_stride3("v_stride"), ("log_decay", vp), ("state", vp), ("lengths", vp)]


class LinearAttentionGrads(ctypes.Structure):
    _fields_ = [("gq", vp), ("gk", vp), ("gv", vp), ("gstate", vp)]


class RotaryParams(ctypes.Structure):
    _fields_ = [("B", i64), ("L", i64), ("H", i32), ("D", i32), ("R", i32), ("interleaved", i32), ("inverse", i32),
                ("scale", f32), *_stride3("x_stride"), ("freq", vp), ("positions", vp), ("pos_sequence", i64),
                ("pos_token", i64)]


class GroupNormParams(ctypes.Structure):
    _fields_ = [("rows", i64), ("D", i32), ("G", i32), ("silu", i32), ("eps", f32), ("x", vp), ("z", vp),
                ("weight", vp), ("bias", vp)]


def declare(L):
    """Argument types of the library's functions for this module."""
    lp, gp, rp, np_ = (ctypes.POINTER(t) for t in (LinearAttentionParams, LinearAttentionGrads, RotaryParams,
                                                   GroupNormParams))
    for name, args, res in (
            ("hyena_linear_attention_workspace_bytes", [i64, i64, i32, i32, i32], i64),
            ("hyena_linear_attention", [lp, vp, vp, i32, vp, i64, vp], i32),
            ("hyena_linear_attention_step", [lp, vp, vp, i32, vp], i32),
            ("hyena_linear_attention_backward_workspace_bytes", [i64, i64] + [i32] * 6, i64),
            ("hyena_linear_attention_backward", [lp, vp, vp, gp, i32, vp, i64, vp], i32),
            ("hyena_rotary", [rp, vp, vp, i32, vp], i32),
            ("hyena_group_norm", [np_, vp, i32, vp], i32),
            ("hyena_group_norm_backward_workspace_bytes", [i64, i32, i32], i64),
            ("hyena_group_norm_backward", [np_, vp, vp, vp, vp, vp, i32, vp, i64, vp], i32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


# ------------------------------------------------------------------ checking

def _heads(t, name, dims, like=None):
    """Checks a tensor [B, L, heads, D] ([B, heads, D] with dims 3) whose heads' values are contiguous; `like`: the
    tensor whose dtype, device and leading sizes it has to share."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (ROCm) tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} has {t.dim()} dimensions, not {dims}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the values of {name}'s heads must be contiguous")
    if like is not None:
        if t.dtype is not like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, not on {like.device}")
        if t.shape[:dims - 2] != like.shape[:dims - 2]:
            raise ValueError(f"{name} shape {tuple(t.shape)} does not start with {tuple(like.shape[:dims - 2])}")


def _strides(s, n):
    """Strides s of sizes n between sequences, tokens and heads; 0 where there is but one."""
    if len(n) == 4:
        return (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)
    return (s[0] if n[0] > 1 else 0, 0, s[1] if n[1] > 1 else 0)


# ---------------------------------------------------------- linear attention

def _attention(q, k, v, log_decay, scale, state, lengths, dims):
    """(io, B, L, H, Dk, Dv, the parameters) of a call; heads as many as q, k or v has most of."""
    import torch
    try:                                              # one expression for a single token's call, where this counts
        t, dev, nq, nk, nv, sq, sk, sv = q.dtype, q.device, q.shape, k.shape, v.shape, q.stride(), k.stride(), v.stride()
        fine = (len(nq) == len(nk) == len(nv) == dims and k.dtype is t and v.dtype is t and q.is_cuda and k.device == dev
                and v.device == dev and sq[-1] == sk[-1] == sv[-1] == 1 and nq[0] == nk[0] == nv[0]
                and (dims == 3 or nq[1] == nk[1] == nv[1]))
    except AttributeError:
        fine = False
    if not fine:                                      # what is wrong, if anything is
        _heads(q, "q", dims)
        _heads(k, "k", dims, q)
        _heads(v, "v", dims, q)
    io = _H._io_of(q)
    B, L = nq[0], nq[1] if dims == 4 else 1
    Hq, Hk, Hv, Dk, Dv = nq[-2], nk[-2], nv[-2], nq[-1], nv[-1]
    if nk[-1] != Dk:
        raise ValueError(f"q and k have heads of {Dk} and {nk[-1]} values")
    H = max(Hq, Hk, Hv)
    if not (Hq and Hk and Hv) or H % Hq or H % Hk or H % Hv:
        raise ValueError(f"{Hq}, {Hk} and {Hv} heads of q, k and v do not divide the most of them")
    if scale is None:
        scale = Dk ** -0.5 if Dk else 0.0
    p = LinearAttentionParams(
        B, L, H, Hq, Hk, Hv, Dk, Dv, scale, 0, q.data_ptr(), k.data_ptr(), v.data_ptr(), *_strides(sq, nq), *_strides(sk, nk),
        *_strides(sv, nv), None if log_decay is None else _take(log_decay, "log_decay", (H,), torch.float32, dev),
        None if state is None else _take(state, "state", (B, H, Dk, Dv), torch.float32, dev),
        None if lengths is None else _take(lengths, "lengths", (B,), torch.int32, dev))
    return io, B, L, H, Dk, Dv, p


def linear_attention_workspace_bytes(B: int, L: int, H: int, Dk: int, Dv: int) -> int:
    return int(_H.lib().hyena_linear_attention_workspace_bytes(B, L, H, Dk, Dv))


def linear_attention(q, k, v, log_decay=None, scale=None, state=None, lengths=None, return_state: bool = False, out=None,
                     state_out=None, workspace=None):
    """o [B, L, H, Dv] of S[t] = exp(log_decay) S[t-1] + k[t] v[t]^T, o[t] =
    scale S[t]^T q[t] for each head.  q [B, L, Hq, Dk], k [B, L, Hk, Dk], v
    [B, L, Hv, Dv]: H, the most of the three, is a multiple of each, and
    neighbouring heads share one where there are fewer.  log_decay [H], not
    positive (None: no decay), state [B, H, Dk, Dv] in float32; lengths int32
    [B]: steps of each sequence, o is zero behind them; scale: Dk^-1/2 by
    default.  Returns o, with return_state (o, S at each sequence's end)."""
    torch = _torch()
    io, B, L, H, Dk, Dv, p = _attention(q, k, v, log_decay, scale, state, lengths, 4)
    dev, shape = q.device, (B, L, H, Dv)
    o = _new(shape, q.dtype, dev) if out is None else out
    op = o.data_ptr() if out is None else _take(out, "out", shape, q.dtype, dev)
    if return_state and state_out is None:
        state_out = _new((B, H, Dk, Dv), torch.float32, dev)
    keep, ws, wsb = _workspace(workspace, linear_attention_workspace_bytes(B, L, H, Dk, Dv),
                               "hyena_linear_attention_workspace_bytes", dev)
    _call("hyena_linear_attention", dev, ctypes.byref(p), op,
          _take(state_out, "state_out", (B, H, Dk, Dv), torch.float32, dev), io, ws, wsb)
    return (o, state_out) if return_state else o


def linear_attention_step(q, k, v, state, log_decay=None, scale=None, out=None):
    """One token for each sequence: q [B, Hq, Dk], k [B, Hk, Dk], v [B, Hv,
    Dv] -> o [B, H, Dv]; state [B, H, Dk, Dv] float32 moves on by one in
    place."""
    import torch
    io, B, _, H, Dk, Dv, p = _attention(q, k, v, log_decay, scale, None, None, 3)
    dev, shape = q.device, (B, H, Dv)
    o = _new(shape, q.dtype, dev) if out is None else out
    op = o.data_ptr() if out is None else _take(out, "out", shape, q.dtype, dev)
    _call("hyena_linear_attention_step", dev, ctypes.byref(p),
          _take(state, "state", (B, H, Dk, Dv), torch.float32, dev), op, io)
    return o


def linear_attention_backward_workspace_bytes(B: int, L: int, H: int, Hq: int, Hk: int, Hv: int, Dk: int, Dv: int) -> int:
    return int(_H.lib().hyena_linear_attention_backward_workspace_bytes(B, L, H, Hq, Hk, Hv, Dk, Dv))


def linear_attention_backward(q, k, v, go, log_decay=None, scale=None, state=None, lengths=None, gstate_out=None,
                              workspace=None) -> dict:
    """Gradients of a loss with dloss/do = go (and dloss/dS = gstate_out at
    the sequences' ends) through linear_attention of the same arguments: a dict
    of gq, gk, gv, summed over the heads that share one, and gstate, None
    without a state.  log_decay is a constant and has none."""
    torch = _torch()
    io, B, L, H, Dk, Dv, p = _attention(q, k, v, log_decay, scale, state, lengths, 4)
    dev, t = q.device, q.dtype
    out = {name: _new(tuple(x.shape), t, dev) for name, x in (("gq", q), ("gk", k), ("gv", v))}
    out["gstate"] = _like(state) if state is not None else None
    g = LinearAttentionGrads(*[x.data_ptr() if x is not None else None for x in out.values()])
    keep, ws, wsb = _workspace(workspace, linear_attention_backward_workspace_bytes(B, L, H, p.Hq, p.Hk, p.Hv, Dk, Dv),
                               "hyena_linear_attention_backward_workspace_bytes", dev)
    _call("hyena_linear_attention_backward", dev, ctypes.byref(p), _take(go, "go", (B, L, H, Dv), t, dev),
          _take(gstate_out, "gstate_out", (B, H, Dk, Dv), torch.float32, dev), ctypes.byref(g), io, ws, wsb)
    return out


# ---------------------------------------------------------- rotary positions

def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, context: int = 4096,
                       turns=(1.0, 32.0), device=None):
    """(freq, scale) for rotary: the angle of one position for each of the
    dim/2 pairs, base^(-2i/dim) as float64 [dim/2], and the factor of its
    outputs.  scaling stretches them for a context `factor` times as long as
    the `context` that a model was trained for: "linear" divides all by factor
    (positions interpolated); "ntk" raises the base to base factor^(dim/(dim-2)),
    which divides the slowest by factor and keeps the fastest; "yarn" keeps
    pairs that turn at least turns[1] times within `context`, divides those
    that turn at most turns[0] times, and gives the scale 0.1 log(factor) + 1
    (to queries and keys alike).  Between them it blends the two linearly in
    the number of turns; a model that was trained with a blend linear in the
    pair's index needs frequencies of its own, which rotary takes as they are."""
    torch = _torch()
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and at least 2, not {dim}")
    if not (base > 0 and factor >= 1 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(0, dim, 2, dtype=torch.float64) / dim
    freq, scale = base ** -i, 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "ntk":
        if dim < 4:
            raise ValueError("ntk scaling takes at least two pairs")
        freq = (base * factor ** (dim / (dim - 2))) ** -i
    elif scaling == "yarn":
        low, high = turns
        if not (context > 0 and high > low):
            raise ValueError("yarn scaling takes a context and two rising numbers of turns")
        keep = ((context * freq / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling != "none":
        raise ValueError(f'scaling must be "none", "linear", "ntk" or "yarn", not {scaling!r}')
    return freq.to(device or "cuda"), scale


def rotary(x, freq, positions=None, scale: float = 1.0, interleaved: bool = False, inverse: bool = False, out=None):
    """x [B, L, H, D] (or a token's [B, H, D]) with the first 2 len(freq)
    values of each head turned in pairs by position * freq and multiplied by
    scale, the others as they are: (a, b) -> scale (a cos - b sin, a sin +
    b cos) of values (i, i + len(freq)), or (2i, 2i + 1) with interleaved.
    freq float64; positions int32 [B, L] or [L] (0, 1, .. by default), for a
    token [B].  inverse turns back: rotary(gy, .., inverse=True) is the
    gradient.  out: x itself (in place) or a contiguous tensor."""
    import torch
    dims = 3 if isinstance(x, torch.Tensor) and x.dim() == 3 else 4
    _heads(x, "x", dims)
    io, dev, n = _H._io_of(x), x.device, x.shape
    B, L, H, D = n[0], n[1] if dims == 4 else 1, n[-2], n[-1]
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise TypeError("freq must be a CUDA (ROCm) tensor of one dimension")
    R = 2 * freq.shape[0]
    if positions is None and dims == 3:
        raise ValueError("a token needs its positions")
    pos, pos_stride = None, (0, 0)
    if positions is not None:
        shape = (B,) if dims == 3 else (L,) if isinstance(positions, torch.Tensor) and positions.dim() == 1 else (B, L)
        pos = _take(positions, "positions", shape, torch.int32, dev)
        pos_stride = (1, 0) if dims == 3 else (L if len(shape) == 2 else 0, 1)
    if out is x:
        op = x.data_ptr()
    elif out is None:
        out = _new(tuple(x.shape), x.dtype, dev)
        op = out.data_ptr()
    else:
        op = _take(out, "out", x.shape, x.dtype, dev)
        if op == x.data_ptr() and not x.is_contiguous():
            raise ValueError("out is x's memory in another layout")
    p = RotaryParams(B, L, H, D, R, int(bool(interleaved)), int(bool(inverse)), scale, *_strides(x.stride(), n),
                     _take(freq, "freq", freq.shape, torch.float64, dev), pos, *pos_stride)
    _call("hyena_rotary", dev, ctypes.byref(p), x.data_ptr(), op, io)
    return out


# ---------------------------------------------------------------- group norm

def _norm_params(x, groups, weight, bias, z, silu, eps):
    torch = _torch()
    io, rows, D = _rows(x, "x")
    dev = x.device
    if groups < 1 or not D or D % groups:
        raise ValueError(f"{D} values to a row do not make {groups} groups")
    if silu and z is not None:
        raise ValueError("silu and z exclude each other")
    return io, rows, D, GroupNormParams(
        rows, D, groups, int(bool(silu)), eps, x.data_ptr(), _take(z, "z", x.shape, x.dtype, dev),
        _take(weight, "weight", (D,), torch.float32, dev), _take(bias, "bias", (D,), torch.float32, dev))


def group_norm(x, groups: int, weight=None, bias=None, z=None, silu: bool = False, eps: float = 1e-5, out=None):
    """Each of the `groups` groups of neighbouring values of x [..., D] (each
    head of a token) normed by itself, m = (x - mean) / sqrt(var + eps) *
    weight + bias, with weight and bias [D] in float32; returns m, with silu
    m * sigmoid(m), or with a gate z [..., D] m * z * sigmoid(z)."""
    io, rows, D, p = _norm_params(x, groups, weight, bias, z, silu, eps)
    y = _like(x) if out is None else out
    yp = y.data_ptr() if out is None else _take(out, "out", x.shape, x.dtype, x.device)
    _call("hyena_group_norm", x.device, ctypes.byref(p), yp, io)
    return y


def group_norm_backward_workspace_bytes(rows: int, D: int, groups: int) -> int:
    return int(_H.lib().hyena_group_norm_backward_workspace_bytes(rows, D, groups))


def group_norm_backward(x, groups: int, gy, weight=None, bias=None, z=None, silu: bool = False, eps: float = 1e-5,
                        workspace=None) -> dict:
    """Gradients of a loss with dloss/dy = gy through group_norm of the same
    arguments: a dict of gx, gweight, gbias (float32, summed over the rows)
    and gz, None where the argument is None."""
    torch = _torch()
    io, rows, D, p = _norm_params(x, groups, weight, bias, z, silu, eps)
    dev = x.device
    out = {"gx": _like(x), "gweight": _new((D,), torch.float32, dev) if weight is not None else None,
           "gbias": _new((D,), torch.float32, dev) if bias is not None else None, "gz": _like(z) if z is not None else None}
    at = {k: t.data_ptr() if t is not None else None for k, t in out.items()}
    need = group_norm_backward_workspace_bytes(rows, D, groups) if weight is not None or bias is not None else 0
    keep, ws, wsb = _workspace(workspace, need, "hyena_group_norm_backward_workspace_bytes", dev)
    _call("hyena_group_norm_backward", dev, ctypes.byref(p), _take(gy, "gy", x.shape, x.dtype, dev), at["gx"],
          at["gweight"], at["gbias"], at["gz"], io, ws, wsb)
    return out
