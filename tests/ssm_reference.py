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


def selective_scan_with_sizes(u, delta, A, Bm, Cm, skip, z, delta_bias, softplus, state, lengths, gy, gstate_out):
    """selective_scan and its gradients in float64 on the arguments' device,
    whole batches at a time: name -> (value, size), size the sum of the sizes
    of the terms that make the value up.  In sizes a state decays with half
    its exponent: a decay exp(-X) of relative error e X is off by
    e X exp(-X) <= e exp(-X / 2)."""
    u, delta, A, Bm, Cm, skip, z, delta_bias, state, gy, gstate_out = (
        t.to(D64) for t in (u, delta, A, Bm, Cm, skip, z, delta_bias, state, gy, gstate_out))
    B, D, L = u.shape
    N, G = A.shape[1], Bm.shape[1]
    ok = torch.ones(B, 1, L, dtype=torch.bool, device=u.device)
    if lengths is not None:
        ok = torch.arange(L, device=u.device).view(1, 1, L) < lengths.view(B, 1, 1)
    put = lambda v, m: torch.where(m, v, torch.zeros((), dtype=D64, device=v.device))  # noqa: E731
    first = lambda v: v.movedim(-1, 0).contiguous()  # noqa: E731: time in front
    pre = delta + delta_bias[:, None]
    sig = 1 / (1 + torch.exp(-pre)) if softplus else torch.ones_like(pre)
    dt = first(put(torch.logaddexp(pre, torch.zeros_like(pre)) if softplus else pre, ok))
    u, z, gy = put(u, ok), put(z, ok), put(gy, ok)
    sz = 1 / (1 + torch.exp(-z))
    gate, slope = z * sz, sz * (1 + z * (1 - sz))
    gg, ut = first(gy * gate), first(u)
    Bm, Cm = first(put(Bm, ok[:, None])), first(put(Cm, ok[:, None]))
    wide = lambda v: v.unsqueeze(2).expand(B, G, D // G, N).reshape(B, D, N)  # noqa: E731
    narrow = lambda v: v.view(B, G, D // G, N).sum(2)  # noqa: E731
    h, hs = [state], [state.abs()]
    y, ys = torch.empty_like(ut), torch.empty_like(ut)
    for t in range(L):
        half = torch.exp(0.5 * dt[t, :, :, None] * A)
        x, C = (dt[t] * ut[t])[..., None] * wide(Bm[t]), wide(Cm[t])
        h.append(half * half * h[-1] + x)
        hs.append(half * hs[-1] + x.abs())
        y[t], ys[t] = (h[-1] * C).sum(-1), (hs[-1] * C.abs()).sum(-1)
    last = (h[-1], hs[-1])
    back = lambda v: v.movedim(0, -1)  # noqa: E731
    y, ys = back(y) + skip[:, None] * u, back(ys) + (skip[:, None] * u).abs()
    q, qs = gstate_out, gstate_out.abs()
    gA, gAs = torch.zeros_like(A), torch.zeros_like(A)
    gB, gBs, gC, gCs = (torch.empty_like(Bm) for _ in range(4))
    gu, gus, gd, gds = (torch.empty_like(ut) for _ in range(4))
    for t in range(L - 1, -1, -1):
        half = torch.exp(0.5 * dt[t, :, :, None] * A)
        Bt, g = wide(Bm[t]), gg[t, :, :, None] * wide(Cm[t])
        ht, hst = h.pop(), hs.pop()
        gC[t], gCs[t] = narrow(ht * gg[t, :, :, None]), narrow(hst * gg[t, :, :, None].abs())
        q, qs = q + g, qs + g.abs()
        v = (dt[t] * ut[t])[..., None]
        gB[t], gBs[t] = narrow(q * v), narrow(qs * v.abs())
        s, ss = (q * Bt).sum(-1), (qs * Bt.abs()).sum(-1)
        q, qs = half * half * q, half * qs
        w, ws = q * h[-1], qs * hs[-1]
        gA += (w * dt[t, :, :, None]).sum(0)
        gAs += (ws * dt[t, :, :, None].abs()).sum(0)
        gd[t], gds[t] = (w * A).sum(-1) + s * ut[t], (ws * A.abs()).sum(-1) + ss * ut[t].abs()
        gu[t], gus[t] = s * dt[t] + skip * gg[t], ss * dt[t].abs() + (skip * gg[t]).abs()
    gd, gds, gg = back(gd) * put(sig, ok), back(gds) * put(sig, ok), back(gg)
    return {"y": (y * gate, ys * gate.abs()), "h": last, "gu": (back(gu), back(gus)), "gdelta": (gd, gds),
            "gA": (gA, gAs), "gB": (back(gB), back(gBs)), "gC": (back(gC), back(gCs)),
            "gskip": ((gg * u).sum((0, 2)), (gg * u).abs().sum((0, 2))),
            # the slope's own terms are at most 1.3 in all
            "gz": (gy * y * slope, 1.3 * gy.abs() * ys), "gdelta_bias": (gd.sum((0, 2)), gds.sum((0, 2))), "gstate": (q, qs)}
