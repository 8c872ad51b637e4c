"""Plain float64 definitions of the state-space block's operators, one step or
one tap after the other, for the tests.  They share no code with the kernels.
Differentiable: gradients come from torch's autograd over these definitions."""
from __future__ import annotations

import torch

D64 = torch.float64


def up(t):
    """A leaf in float64 on the CPU, or None."""
    return None if t is None else t.detach().to("cpu", D64 if t.is_floating_point() else torch.int64)


def silu(p):
    return p / (1 + torch.exp(-p))


def clamp_lengths(lengths, B, L):
    return [L] * B if lengths is None else [min(max(int(n), 0), L) for n in lengths.tolist()]


def short_conv(x, w, bias=None, use_silu=False, state=None, lengths=None):
    """(y, the last T-1 inputs) of x [B, D, L]."""
    B, D, L = x.shape
    T = w.shape[1]
    ys, lasts = [], []
    for b, n in enumerate(clamp_lengths(lengths, B, L)):
        front = state[b] if state is not None else torch.zeros(D, T - 1, dtype=D64)
        xe = torch.cat((front, x[b, :, :n]), 1)
        p = torch.zeros(D, n, dtype=D64)
        for j in range(T):
            p = p + w[:, j:j + 1] * xe[:, T - 1 - j:T - 1 - j + n]
        if bias is not None:
            p = p + bias[:, None]
        y = silu(p) if use_silu else p
        ys.append(torch.cat((y, torch.zeros(D, L - n, dtype=D64)), 1))
        lasts.append(xe[:, n:])
    return torch.stack(ys), torch.stack(lasts)


def selective_scan(u, delta, A, Bm, Cm, skip=None, z=None, delta_bias=None, softplus=True, state=None, lengths=None):
    """(y, h at the ends) of u [B, D, L]."""
    B, D, L = u.shape
    N, G = A.shape[1], Bm.shape[1]
    ys, hs = [], []
    for b, n in enumerate(clamp_lengths(lengths, B, L)):
        h = state[b] if state is not None else torch.zeros(D, N, dtype=D64)
        cols = []
        for t in range(n):
            x = delta[b, :, t] + (delta_bias if delta_bias is not None else 0)
            dt = torch.logaddexp(x, torch.zeros_like(x)) if softplus else x
            Bt = Bm[b, :, :, t].repeat_interleave(D // G, 0)
            Ct = Cm[b, :, :, t].repeat_interleave(D // G, 0)
            h = torch.exp(dt[:, None] * A) * h + (dt * u[b, :, t])[:, None] * Bt
            y = (Ct * h).sum(1)
            if skip is not None:
                y = y + skip * u[b, :, t]
            cols.append(y * silu(z[b, :, t]) if z is not None else y)
        cols += [torch.zeros(D, dtype=D64)] * (L - n)
        ys.append(torch.stack(cols, 1))
        hs.append(h)
    return torch.stack(ys), torch.stack(hs)


def rms_norm(s, weight, eps):
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * weight


def quantize(v, rows):
    """Codes (as float64 values) and scales of v [R, K] (float32 values held in
    float64), the scale rounded to float32 and the quotient rounded once."""
    R, K = v.shape
    codes, scales = torch.empty_like(v), torch.empty(-(-R // rows), -(-K // 128), dtype=D64)
    for i in range(scales.shape[0]):
        for k in range(scales.shape[1]):
            blk = v[rows * i:rows * (i + 1), 128 * k:128 * (k + 1)]
            top = blk.abs().max()
            s = (top / 448).float().double() if top > 0 else torch.ones((), dtype=D64)
            scales[i, k] = s
            codes[rows * i:rows * (i + 1), 128 * k:128 * (k + 1)] = (blk / s).float().to(torch.float8_e4m3fn).double()
    return codes, scales


def scaled_matmul(q, scales, wq, wscales, bias=None):
    """(the product [M, N], the sum of its terms' sizes)."""
    left = q * scales.repeat_interleave(128, 1)[:, :q.shape[1]]
    right = wq * wscales.repeat_interleave(128, 0)[:wq.shape[0]].repeat_interleave(128, 1)[:, :wq.shape[1]]
    out, size = left @ right.t(), left.abs() @ right.abs().t()
    if bias is not None:
        out, size = out + bias, size + bias.abs()
    return out, size
