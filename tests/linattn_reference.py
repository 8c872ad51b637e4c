"""Plain float64 definitions of the linear-attention block's operators, one
token after the other, for the tests.  They share no code with the kernels.

Each result comes as (value, size), size the sum of the sizes of the terms that
make the value up.  In sizes a state decays with half its exponent: a decay
exp(-X) of relative error e X is off by e X exp(-X) <= e exp(-X / 2)."""
from __future__ import annotations

import torch

from tests.ssm_reference import D64, clamp_lengths


def linear_attention(q, k, v, log_decay=None, scale=None, state=None, lengths=None, go=None, gstate_out=None):
    """{"o", "state"} and, with go, {"gq", "gk", "gv", "gstate"} of q [B, L, Hq, Dk], k [B, L, Hk, Dk], v [B, L, Hv, Dv], on q's device."""
    up = lambda t: None if t is None else t.detach().to(D64)  # noqa: E731
    q, k, v, log_decay, state, go, gstate_out = map(up, (q, k, v, log_decay, state, go, gstate_out))
    B, L, Dk, Dv = q.shape[0], q.shape[1], q.shape[-1], v.shape[-1]
    heads = (q.shape[2], k.shape[2], v.shape[2])
    H = max(heads)
    scale = Dk ** -0.5 if scale is None else scale
    dev = q.device
    n = torch.tensor(clamp_lengths(lengths, B, L), device=dev)
    inside = torch.arange(L, device=dev)[:, None] < n                      # [L, B]

    def first(x):                                                           # [L, B, H, D], zeros behind a length
        x = torch.where(inside.t()[:, :, None, None], x, torch.zeros((), dtype=D64, device=dev))
        return x.repeat_interleave(H // x.shape[2], 2).transpose(0, 1).contiguous()

    q, k, v = first(q), first(k), first(v)
    g = log_decay if log_decay is not None else torch.zeros(H, dtype=D64, device=dev)
    lam, half = (torch.where(inside[..., None], torch.exp(x), torch.ones((), dtype=D64, device=dev))[..., None, None] for x in (g, 0.5 * g))
    zeros = torch.zeros(B, H, Dk, Dv, dtype=D64, device=dev)
    S = state.clone() if state is not None else zeros.clone()
    Z = S.abs()
    go = first(go) if go is not None else None
    o, oz = torch.empty_like(v), torch.empty_like(v)
    gq, gqz = torch.empty_like(q), torch.empty_like(q)
    for t in range(L):
        x = k[t][..., :, None] * v[t][..., None, :]
        x = torch.where(inside[t][:, None, None, None], x, zeros)
        S, Z = lam[t] * S + x, half[t] * Z + x.abs()
        o[t], oz[t] = scale * (S * q[t][..., :, None]).sum(-2), abs(scale) * (Z * q[t].abs()[..., :, None]).sum(-2)
        if go is not None:
            gq[t], gqz[t] = scale * (S * go[t][..., None, :]).sum(-1), abs(scale) * (Z * go[t].abs()[..., None, :]).sum(-1)
    where = inside[..., None, None]
    back = lambda x: torch.where(where, x, torch.zeros((), dtype=D64, device=dev)).transpose(0, 1)  # noqa: E731
    out = {"o": (back(o), back(oz)), "state": (S, Z)}
    if go is None:
        return out
    G = gstate_out.clone() if gstate_out is not None else zeros.clone()
    W = G.abs()
    gk, gkz, gv, gvz = torch.empty_like(k), torch.empty_like(k), torch.empty_like(v), torch.empty_like(v)
    for t in range(L - 1, -1, -1):
        x = scale * q[t][..., :, None] * go[t][..., None, :]
        G, W = G + x, W + x.abs()
        gk[t], gkz[t] = (G * v[t][..., None, :]).sum(-1), (W * v[t].abs()[..., None, :]).sum(-1)
        gv[t], gvz[t] = (G * k[t][..., :, None]).sum(-2), (W * k[t].abs()[..., :, None]).sum(-2)
        G, W = lam[t] * G, half[t] * W
    fold = lambda x, m: back(x).reshape(B, L, m, H // m, -1).sum(3)  # noqa: E731
    out.update({name: (fold(x, m), fold(z, m)) for name, x, z, m in (("gq", gq, gqz, heads[0]), ("gk", gk, gkz, heads[1]),
                                                                    ("gv", gv, gvz, heads[2]))})
    out["gstate"] = (G, W)
    return out


def linear_attention_by_sums(q, k, v, log_decay, scale, state, lengths):
    """o and the state as the double sum over pairs of tokens, differentiable; all heads alike."""
    B, L, H, _ = q.shape
    os, ss = [], []
    t = torch.arange(L, dtype=D64)
    for b, n in enumerate(clamp_lengths(lengths, B, L)):
        qb, kb, vb = (x[b, :n].transpose(0, 1) for x in (q, k, v))          # [H, n, D]
        g = log_decay[:, None, None]
        w = torch.exp(g * (t[:n, None] - t[None, :n]).clamp(min=0)) * (t[:n, None] >= t[None, :n])
        o = (qb @ kb.transpose(1, 2) * w) @ vb + torch.exp(g * (t[:n, None] + 1)) * (qb @ state[b])
        os.append(torch.cat((scale * o.transpose(0, 1), torch.zeros(L - n, H, v.shape[-1], dtype=D64))))
        ss.append(torch.exp(g * n) * state[b] + (kb * torch.exp(g * (n - 1 - t[:n, None]))).transpose(1, 2) @ vb)
    return torch.stack(os), torch.stack(ss)


def rotary(x, freq, positions, scale=1.0, interleaved=False, inverse=False):
    """x [B, L, H, D] in float64, positions [B, L]."""
    R = 2 * freq.shape[0]
    out = x.clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        angle = (positions.to(D64) * freq[i] * (-1 if inverse else 1))[..., None]
        out[..., a] = scale * (x[..., a] * torch.cos(angle) - x[..., b] * torch.sin(angle))
        out[..., b] = scale * (x[..., a] * torch.sin(angle) + x[..., b] * torch.cos(angle))
    return out


def group_norm(x, groups, weight=None, bias=None, z=None, silu=False, eps=1e-5):
    rows, D = x.shape
    f = x.view(rows, groups, D // groups)
    d = f - f.mean(-1, keepdim=True)
    m = (d / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)).reshape(rows, D)
    if weight is not None:
        m = m * weight
    if bias is not None:
        m = m + bias
    act = lambda p: p / (1 + torch.exp(-p))  # noqa: E731
    return act(m) if silu else m * act(z) if z is not None else m
