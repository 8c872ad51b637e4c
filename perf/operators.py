"""Measured cases of the state-space block's operators.

The block: a residual addition with a root-mean-square norm (its output in the
I/O dtype, or in 8 bits with a scale for each 128 values), a matrix product of
8-bit operands, a short causal convolution, and a selective state-space scan.
Each operator comes with its form for single tokens where it carries a state,
and with its backward pass where a training step needs one.

    short convolution   p[t] = bias + sum_j w[j] x[t-j],  y = p or p * sigmoid(p)
    selective scan      dt = softplus(delta + delta_bias),
                        h[t] = exp(dt[t] A) h[t-1] + dt[t] u[t] B[t],
                        y[t] = (sum_n C[t] h[t] + skip u[t]) * z[t] sigmoid(z[t])
    norm                s = x + residual,  y = s / sqrt(mean(s^2) + eps) * weight
    8-bit values        scale = max|v| / 448 over a block, q = e4m3(v / scale)
    8-bit product       out[m][n] = sum_k (q scale)[m][k] (wq wscale)[n][k] + bias

`run` computes the plain forms with elementary torch operations, or, where
`own` is set, calls this package.  `exact` is the same in float64.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
E4M3_MAX = 448.0


def listed():
    return [
        # A batch of ragged, right-padded prompts read by the short convolution, which leaves each sequence's
        # last inputs behind for the single-token steps that follow.
        dict(name="conv_prompts", op="conv", dtype="bf16", B=8, D=1536, L=2048, T=4, silu=True, state=False, lengths=True),
        # The convolution's gradients in a training step.
        dict(name="conv_backward", op="conv_bwd", dtype="bf16", B=8, D=1536, L=2048, T=4, silu=True, state=False, lengths=False),
        # One new token for each of 16 sequences: the smallest call, all latency.
        dict(name="conv_token", op="conv_step", dtype="bf16", B=16, D=1536, T=4, silu=True),
        # The scan in a training step's forward pass: many rows, gated.
        dict(name="scan_training", op="scan", dtype="bf16", B=8, D=1536, L=2048, N=16, G=1, z=True, state=False, lengths=False),
        # One long sequence (the 64K-token shape) in fp32: few rows, so the time axis has to be split.
        dict(name="scan_long", op="scan", dtype="fp32", B=1, D=768, L=65536, N=16, G=1, z=True, state=True, lengths=False),
        # The scan's gradients in a training step.
        dict(name="scan_backward", op="scan_bwd", dtype="bf16", B=4, D=1536, L=2048, N=16, G=1, z=True, state=False, lengths=False),
        # One new token for each of 128 sequences: the state's traffic.
        dict(name="scan_token", op="scan_step", dtype="bf16", B=128, D=1536, N=16, G=1, z=True),
        # Residual addition and norm before a block, activations of a training step.
        dict(name="norm_residual", op="norm", dtype="bf16", rows=16384, D=768, residual=True),
        # The same in front of an 8-bit product, with an odd number of rows.
        dict(name="norm_8bit", op="norm_q", dtype="bf16", rows=8191, D=2048, residual=True),
        # The norm's gradients in a training step.
        dict(name="norm_backward", op="norm_bwd", dtype="bf16", rows=16384, D=768, residual=True),
        # The projection of one token for each of 16 sequences: the weights' traffic.
        dict(name="product_tokens", op="product", dtype="bf16", M=16, N=4096, K=2048, from_values=False, channel_major=False, bias=False),
        # The projection of prompts, from bf16 activations (cast to 8 bits in the call) to channel-major streams.
        dict(name="product_prompts", op="product", dtype="bf16", M=8192, N=8192, K=2048, from_values=True, channel_major=True, bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "conv_step", "scan", "scan_bwd", "scan_step", "norm", "norm_q", "norm_bwd", "product"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp32"]))
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("conv", "conv_bwd"):
        B, D, L = _log(rng, 1, 16), _log(rng, 16, 4096), _log(rng, 1, 65536)
        L = max(1, min(L, 25_000_000 // (B * D)))
        c.update(B=B, D=D, L=L, T=rng.choice([2, 3, 4, 4, 4, 7, 16]), silu=yes(), state=yes(), lengths=yes())
    elif op == "conv_step":
        c.update(B=_log(rng, 1, 512), D=_log(rng, 16, 8192), T=rng.choice([2, 3, 4, 4, 4, 7, 16]), silu=yes())
    elif op in ("scan", "scan_bwd"):
        B, N, L = _log(rng, 1, 16), rng.choice([1, 4, 8, 11, 16, 16, 16, 32, 64]), _log(rng, 1, 65536)
        G = rng.choice([1, 1, 2, 4])
        D = G * _log(rng, 4, 1024)
        most = 400_000_000 if op == "scan" else 200_000_000
        L = max(1, min(L, most // (B * D * N)))
        c.update(B=B, D=D, L=L, N=N, G=G, z=yes(), state=yes(), lengths=yes())
    elif op == "scan_step":
        G = rng.choice([1, 1, 2, 4])
        c.update(B=_log(rng, 1, 256), D=G * _log(rng, 16, 2048), N=rng.choice([1, 4, 8, 11, 16, 16, 16, 32, 64]), G=G, z=yes())
    elif op in ("norm", "norm_q", "norm_bwd"):
        D = _log(rng, 16, 16384)
        rows = max(1, min(_log(rng, 1, 65536), 25_000_000 // D))
        c.update(rows=rows, D=D, residual=yes())
    else:
        N, K = _log(rng, 16, 8192), 16 * _log(rng, 4, 256)
        M = max(1, min(_log(rng, 1, 16384), 100_000_000_000 // (N * K)))
        c.update(M=M, N=N, K=K, from_values=yes(), channel_major=yes(), bias=yes())
    return c


# ------------------------------------------------------------------ inputs

def _conv_inputs(c, r, t):
    B, D, T = c["B"], c["D"], c["T"]
    s = {"w": r(D, T) / math.sqrt(T), "bias": 0.1 * r(D)}
    if c["op"] == "conv_step":
        s.update(x=r(B, D).to(t), state=r(B, D, T - 1).to(t))
        return s
    s.update(x=r(B, D, c["L"]).to(t), state=r(B, D, T - 1).to(t) if c["state"] else None)
    if c["op"] == "conv_bwd":
        s.update(gy=r(B, D, c["L"]).to(t), gstate_out=r(B, D, T - 1).to(t) if c["state"] else None)
    return s


def _scan_inputs(c, r, u, t):
    B, D, N, G = c["B"], c["D"], c["N"], c["G"]
    tail = () if c["op"] == "scan_step" else (c["L"],)
    step = torch.exp(u(D) * math.log(100.0) + math.log(1e-3))  # time steps of 0.001 to 0.1
    s = {
        "u": r(B, D, *tail).to(t),
        "delta": (0.5 * r(B, D, *tail)).to(t),
        "A": -torch.arange(1, N + 1, device=DEV, dtype=torch.float32) * (0.75 + 0.5 * u(D, 1)),
        "Bm": r(B, G, N, *tail).to(t),
        "Cm": r(B, G, N, *tail).to(t),
        "skip": r(D),
        "z": r(B, D, *tail).to(t) if c["z"] else None,
        "delta_bias": step + torch.log(-torch.expm1(-step)),  # softplus of it is the step
        "state": r(B, D, N) if c["op"] == "scan_step" or c["state"] else None,
    }
    if c["op"] == "scan_bwd":
        s.update(gy=r(B, D, *tail).to(t), gstate_out=r(B, D, N) if c["state"] else None)
    return s


def _blocks(v, rows):
    """v [R, K] in blocks of `rows` x 128, zeros behind its edges: [R', rows, K', 128]."""
    R, K = v.shape
    pad = torch.nn.functional.pad(v, (0, -K % 128, 0, -R % rows))
    return pad.reshape(-(-R // rows), rows, -(-K // 128), 128)


def _spread(scales, R, K, rows):
    """A block's scale at each of its values: [R, K]."""
    return scales.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :K]


def _quantized(v, rows):
    """Codes and scales of v [R, K]: one scale for each block of `rows` x 128."""
    R, K = v.shape
    top = _blocks(v.abs(), rows).amax((1, 3))
    # divided by a tensor: a division by a number is done as a product with its reciprocal, another value
    scales = torch.where(top > 0, top / torch.full_like(top, E4M3_MAX), torch.ones_like(top))
    return (v / _spread(scales, R, K, rows)).to(torch.float32).to(torch.float8_e4m3fn), scales.to(torch.float32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *n: torch.randn(*n, generator=g, device=DEV)  # noqa: E731
    u = lambda *n: torch.rand(*n, generator=g, device=DEV)  # noqa: E731
    c, t = case, TYPES[case["dtype"]]
    op = c["op"]
    if op.startswith("conv"):
        s = _conv_inputs(c, r, t)
    elif op.startswith("scan"):
        s = _scan_inputs(c, r, u, t)
    elif op.startswith("norm"):
        s = {"x": r(c["rows"], c["D"]).to(t), "residual": (2 * r(c["rows"], c["D"])).to(t) if c["residual"] else None,
             "weight": 1 + 0.2 * r(c["D"])}
        if op == "norm_bwd":
            s.update(gy=r(c["rows"], c["D"]).to(t), gs=r(c["rows"], c["D"]).to(t) if c["residual"] else None)
    else:
        x = r(c["M"], c["K"]) * torch.exp(r(c["M"], 1))
        wq, wscales = _quantized(r(c["N"], c["K"]) / math.sqrt(c["K"]), 128)
        s = {"wq": wq, "wscales": wscales, "bias": r(c["N"]) if c["bias"] else None}
        if c["from_values"]:
            s["x"] = x.to(t)
        else:
            s["q"], s["scales"] = _quantized(x, 1)
    if op in ("conv", "conv_bwd", "scan", "scan_bwd"):
        s["lengths"] = None
        if c["lengths"]:  # right-padded prompts: the padding holds whatever was there
            n = (u(c["B"]) * (c["L"] + 1)).to(torch.int32).clamp_(max=c["L"])
            n[0] = c["L"]
            s["lengths"] = n
    s["case"] = c
    return s


# ------------------------------------------------------------- plain forms

def _inside(s, L):
    """[B, 1, L]: the positions before each sequence's length."""
    at = torch.arange(L, device=DEV)
    n = s["lengths"]
    return at.view(1, 1, L) < (n.view(-1, 1, 1) if n is not None else L)


def _conv_parts(s, c):
    """Inputs with the carried ones in front [B, D, T-1+L] (zeros behind a length), and their windows [B, D, L, T]."""
    x, T = s["x"].float(), c["T"]
    x = torch.where(_inside(s, c["L"]), x, torch.zeros_like(x))
    front = s["state"].float() if s["state"] is not None else x.new_zeros(c["B"], c["D"], T - 1)
    xe = torch.cat((front, x), -1)
    return xe, xe.unfold(-1, T, 1).flip(-1)


def _conv(s, c):
    t, T = s["x"].dtype, c["T"]
    xe, windows = _conv_parts(s, c)
    p = (windows * s["w"][:, None, :]).sum(-1) + s["bias"][:, None]
    y = p * torch.sigmoid(p) if c["silu"] else p
    y = torch.where(_inside(s, c["L"]), y, torch.zeros_like(y))
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((c["B"],), c["L"], device=DEV)
    at = (n.view(-1, 1, 1) + torch.arange(T - 1, device=DEV)).expand(-1, c["D"], -1)
    return y.to(t), torch.gather(xe, 2, at).to(t)


def _conv_bwd(s, c):
    t, T, L = s["x"].dtype, c["T"], c["L"]
    _, windows = _conv_parts(s, c)
    gp = s["gy"].float()
    if c["silu"]:
        p = (windows * s["w"][:, None, :]).sum(-1) + s["bias"][:, None]
        sig = torch.sigmoid(p)
        gp = gp * sig * (1 + p * (1 - sig))
    gp = torch.where(_inside(s, L), gp, torch.zeros_like(gp))
    gw = (windows * gp[..., None]).sum((0, 2), dtype=torch.float64).float()
    gbias = gp.sum((0, 2), dtype=torch.float64).float()
    gxe = (torch.nn.functional.pad(gp, (T - 1, T - 1)).unfold(-1, T, 1) * s["w"][:, None, :]).sum(-1)
    if s["gstate_out"] is not None:
        n = s["lengths"].long() if s["lengths"] is not None else torch.full((c["B"],), L, device=DEV)
        at = (n.view(-1, 1, 1) + torch.arange(T - 1, device=DEV)).expand(-1, c["D"], -1)
        gxe = gxe.scatter_add(2, at, s["gstate_out"].float())
    return gxe[..., T - 1:].to(t), gw, gbias, gxe[..., :T - 1].to(t) if s["state"] is not None else None


def _conv_step(s, c):
    t = s["x"].dtype
    xe = torch.cat((s["state"], s["x"][..., None]), -1)
    p = (xe.float().flip(-1) * s["w"]).sum(-1) + s["bias"]
    y = p * torch.sigmoid(p) if c["silu"] else p
    s["state"].copy_(xe[..., 1:])
    return y.to(t), s["state"]


def _softplus(x):
    return torch.relu(x) + torch.log1p(torch.exp(-x.abs()))


def _prefix(a, b):
    """h[t] = a[t] h[t-1] + b[t] along the last axis, by pairs."""
    L = b.shape[-1]
    if L == 1:
        return b
    m = L // 2 * 2
    odd = _prefix(a[..., 1:m:2] * a[..., 0:m:2], a[..., 1:m:2] * b[..., 0:m:2] + b[..., 1:m:2])
    h = torch.empty_like(b)
    h[..., 0] = b[..., 0]
    h[..., 1:m:2] = odd
    h[..., 2::2] = a[..., 2::2] * odd[..., :(L - 1) // 2] + b[..., 2::2]
    return h


def _scan_parts(s, c):
    """u, dt, z, B, C with zeros behind a length (B, C [B, D, N, L]), the decays and the states [B, D, N, L]."""
    L, per = c["L"], c["D"] // c["G"]
    ok = _inside(s, L)
    zero = torch.zeros((), device=DEV)
    u = torch.where(ok, s["u"].float(), zero)
    pre = torch.where(ok, s["delta"].float() + s["delta_bias"][:, None], zero)
    dt = torch.where(ok, _softplus(pre), zero)
    z = torch.where(ok, s["z"].float(), zero) if s["z"] is not None else None
    Bm = torch.where(ok[:, :, None], s["Bm"].float(), zero).repeat_interleave(per, 1)
    Cm = torch.where(ok[:, :, None], s["Cm"].float(), zero).repeat_interleave(per, 1)
    a = torch.exp(dt[:, :, None] * s["A"][:, :, None])
    b = (dt * u)[:, :, None] * Bm
    if s["state"] is not None:
        b[..., 0] += a[..., 0] * s["state"]
    return u, pre, dt, z, Bm, Cm, a, _prefix(a, b)


def _scan(s, c):
    u, _, _, z, _, Cm, _, h = _scan_parts(s, c)
    y = (h * Cm).sum(2) + s["skip"][:, None] * u
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y.to(s["u"].dtype), h[..., -1].contiguous()


def _scan_bwd(s, c):
    t, B, D, L, N, G = s["u"].dtype, c["B"], c["D"], c["L"], c["N"], c["G"]
    u, pre, dt, z, Bm, Cm, a, h = _scan_parts(s, c)
    ok = _inside(s, L)
    gy = torch.where(ok, s["gy"].float(), torch.zeros((), device=DEV))
    gz = None
    if z is not None:
        sig = torch.sigmoid(z)
        gz = (gy * ((h * Cm).sum(2) + s["skip"][:, None] * u) * sig * (1 + z * (1 - sig))).to(t)
        gy = gy * z * sig
    late = torch.zeros_like(h)  # the loss's gradient with respect to h[t], before the later steps' share
    late += gy[:, :, None] * Cm
    if s["gstate_out"] is not None:
        late[..., -1] += s["gstate_out"]
    after = torch.cat((a[..., 1:], torch.zeros_like(a[..., :1])), -1)
    gh = _prefix(after.flip(-1), late.flip(-1)).flip(-1)
    before = torch.cat((s["state"][..., None] if s["state"] is not None else torch.zeros_like(h[..., :1]), h[..., :-1]), -1)
    ga = gh * a * before  # times dt: A's gradient; times A: dt's
    gb = (gh * Bm).sum(2)
    gdt = torch.where(ok, (ga * s["A"][:, :, None]).sum(2) + gb * u, torch.zeros((), device=DEV))
    gdelta = gdt * torch.sigmoid(pre)
    of_group = lambda v: v.reshape(B, G, D // G, N, L).sum(2).to(t)  # noqa: E731
    return {
        "gu": (gb * dt + s["skip"][:, None] * gy).to(t),
        "gdelta": gdelta.to(t),
        "gA": (ga * dt[:, :, None]).sum((0, 3), dtype=torch.float64).float(),
        "gB": of_group(gh * (dt * u)[:, :, None]),
        "gC": of_group(h * gy[:, :, None]),
        "gskip": (gy * u).sum((0, 2), dtype=torch.float64).float(),
        "gz": gz,
        "gdelta_bias": gdelta.sum((0, 2), dtype=torch.float64).float(),
        "gstate": a[..., 0] * gh[..., 0] if s["state"] is not None else None,
    }


def _scan_step(s, c):
    t, per = s["u"].dtype, c["D"] // c["G"]
    u = s["u"].float()
    dt = _softplus(s["delta"].float() + s["delta_bias"])
    Bm, Cm = s["Bm"].float().repeat_interleave(per, 1), s["Cm"].float().repeat_interleave(per, 1)
    h = torch.exp(dt[..., None] * s["A"]) * s["state"] + (dt * u)[..., None] * Bm
    s["state"].copy_(h)
    y = (h * Cm).sum(-1) + s["skip"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(t), s["state"]


def _norm(s, c):
    t = s["x"].dtype
    v = (s["x"].float() + s["residual"].float()).to(t) if s["residual"] is not None else s["x"]
    f = v.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["weight"]
    carried = (v,) if s["residual"] is not None else ()
    if c["op"] == "norm":
        return (y.to(t), *carried)
    q, scales = _quantized(y, 1)
    return (q, scales, *carried)


def _norm_bwd(s, c):
    t = s["x"].dtype
    f, gy = s["x"].float(), s["gy"].float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    gw = (gy * f * r).sum(0, dtype=torch.float64).float()
    g = gy * s["weight"]
    gx = r * (g - f * r * (g * f * r).mean(-1, keepdim=True))
    if s["gs"] is not None:
        gx = gx + s["gs"].float()
    return gx.to(t), gw


def _product(s, c):
    q, scales = (s["q"], s["scales"]) if "q" in s else _quantized(s["x"].float(), 1)
    left = q.float() * _spread(scales, c["M"], c["K"], 1)
    right = s["wq"].float() * _spread(s["wscales"], c["N"], c["K"], 128)
    out = left @ right.t()
    if s["bias"] is not None:
        out = out + s["bias"]
    return (out.t().contiguous() if c["channel_major"] else out).to(TYPES[c["dtype"]])


PLAIN = {"conv": _conv, "conv_bwd": _conv_bwd, "conv_step": _conv_step, "scan": _scan, "scan_bwd": _scan_bwd,
         "scan_step": _scan_step, "norm": _norm, "norm_q": _norm, "norm_bwd": _norm_bwd, "product": _product}


def _values(q, scales):
    """What 8-bit codes stand for, in the dtype that holds a code's steps."""
    return (q.float() * _spread(scales, q.shape[0], q.shape[1], 1)).to(torch.bfloat16)


# ---------------------------------------------------------- this package's

def _run_own(s, c):
    import hyena_long_conv_amd as H
    op = c["op"]
    if op == "conv":
        return H.short_conv(s["x"], s["w"], s["bias"], silu=c["silu"], state=s["state"], lengths=s["lengths"], return_state=True)
    if op == "conv_bwd":
        return H.short_conv_backward(s["x"], s["w"], s["gy"], s["bias"], silu=c["silu"], state=s["state"], lengths=s["lengths"],
                                     gstate_out=s["gstate_out"])
    if op == "conv_step":
        return H.short_conv_step(s["x"], s["w"], s["state"], s["bias"], silu=c["silu"]), s["state"]
    if op == "scan":
        return H.selective_scan(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], skip=s["skip"], z=s["z"], delta_bias=s["delta_bias"],
                                softplus=True, state=s["state"], lengths=s["lengths"], return_state=True)
    if op == "scan_bwd":
        return H.selective_scan_backward(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["gy"], skip=s["skip"], z=s["z"],
                                         delta_bias=s["delta_bias"], softplus=True, state=s["state"], lengths=s["lengths"],
                                         gstate_out=s["gstate_out"])
    if op == "scan_step":
        return H.selective_scan_step(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["state"], skip=s["skip"], z=s["z"],
                                     delta_bias=s["delta_bias"], softplus=True), s["state"]
    if op == "norm":
        out = H.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return out if s["residual"] is not None else (out,)
    if op == "norm_q":
        return H.rms_norm_quantized(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    if op == "norm_bwd":
        return H.rms_norm_backward(s["x"], s["weight"], s["gy"], gs=s["gs"], eps=EPS)
    q, scales = (s["q"], s["scales"]) if "q" in s else H.quantize(s["x"])
    return H.scaled_matmul(q, scales, s["wq"], s["wscales"], bias=s["bias"], out_dtype=TYPES[c["dtype"]],
                           channel_major=c["channel_major"])


def run(state):
    c = state["case"]
    out = _run_own(state, c) if own else PLAIN[c["op"]](state, c)
    if c["op"] == "norm_q":
        return (_values(out[0], out[1]), *out[1:])
    return out


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    op = c["op"]
    if op.startswith("conv"):
        n, rest = c["B"] * c["D"], 4 * c["D"] * (c["T"] + 1)
        if op == "conv_step":
            return {"bytes": e * n * (2 + 2 * (c["T"] - 1)) + rest, "flops": n * (2 * c["T"] + 4)}
        n_t = n * c["L"]
        carried = e * n * (c["T"] - 1)
        if op == "conv":
            return {"bytes": e * n_t * 2 + carried * (2 if c["state"] else 1) + rest, "flops": n_t * (2 * c["T"] + 4)}
        return {"bytes": e * n_t * 3 + carried * (3 if c["state"] else 0) + 2 * rest, "flops": n_t * (6 * c["T"] + 12)}
    if op.startswith("scan"):
        rows, N, L = c["B"] * c["D"], c["N"], c.get("L", 1)
        n_t, bc = rows * L, 2 * c["B"] * c["G"] * N * L
        gate = 1 if c["z"] else 0
        rest = 4 * c["D"] * (N + 2)
        if op == "scan_step":
            return {"bytes": e * (n_t * (3 + gate) + bc) + 8 * rows * N + rest, "flops": n_t * (7 * N + 20)}
        if op == "scan":
            return {"bytes": e * (n_t * (3 + gate) + bc) + 4 * rows * N * (2 if c["state"] else 1) + rest, "flops": n_t * (7 * N + 20)}
        return {"bytes": e * (n_t * (5 + 2 * gate) + 2 * bc) + 4 * rows * N * (3 if c["state"] else 0) + 2 * rest, "flops": n_t * (22 * N + 40)}
    if op.startswith("norm"):
        n, more = c["rows"] * c["D"], 2 if c["residual"] else 0
        if op == "norm":
            return {"bytes": e * n * (2 + more) + 4 * c["D"], "flops": 5 * n}
        if op == "norm_q":
            return {"bytes": e * n * (1 + more) + n + 4 * c["rows"] * -(-c["D"] // 128) + 4 * c["D"], "flops": 8 * n}
        return {"bytes": e * n * (3 + more // 2) + 8 * c["D"], "flops": 12 * n}
    M, N, K = c["M"], c["N"], c["K"]
    kb = -(-K // 128)
    left = e * M * K if c["from_values"] else M * K + 4 * M * kb
    return {"bytes": left + N * K + 4 * -(-N // 128) * kb + e * M * N + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}


# ---------------------------------------------------------------- 64 bits

def _exact_conv(s, c):
    d = torch.float64
    B, D, L, T = c["B"], c["D"], c["L"], c["T"]
    n = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    w, bias = s["w"].to(d), s["bias"].to(d)
    back = c["op"] == "conv_bwd"
    y = torch.zeros(B, D, L, dtype=d, device=DEV)
    last = torch.zeros(B, D, T - 1, dtype=d, device=DEV)
    gx, gfirst, gw, gbias = torch.zeros_like(y), torch.zeros_like(last), torch.zeros_like(w), torch.zeros_like(bias)
    for b in range(B):
        m = n[b]
        xe = torch.zeros(D, T - 1 + m, dtype=d, device=DEV)
        if s["state"] is not None:
            xe[:, :T - 1] = s["state"][b].to(d)
        xe[:, T - 1:] = s["x"][b, :, :m].to(d)
        last[b] = xe[:, m:]
        p = bias[:, None].repeat(1, m)
        for j in range(T):
            p += w[:, j:j + 1] * xe[:, T - 1 - j:T - 1 - j + m]
        sig = 1 / (1 + torch.exp(-p))
        y[b, :, :m] = p * sig if c["silu"] else p
        if back:
            gp = s["gy"][b, :, :m].to(d)
            if c["silu"]:
                gp = gp * (sig + p * sig * (1 - sig))
            gxe = torch.zeros_like(xe)
            for j in range(T):
                gxe[:, T - 1 - j:T - 1 - j + m] += w[:, j:j + 1] * gp
                gw[:, j] += (gp * xe[:, T - 1 - j:T - 1 - j + m]).sum(-1)
            gbias += gp.sum(-1)
            if s["gstate_out"] is not None:
                gxe[:, m:] += s["gstate_out"][b].to(d)
            gfirst[b], gx[b, :, :m] = gxe[:, :T - 1], gxe[:, T - 1:]
    if back:
        return gx, gw, gbias, gfirst if s["state"] is not None else None
    return y, last


def _exact_conv_step(s, c):
    d = torch.float64
    T = c["T"]
    p = s["bias"].to(d) + s["w"][:, 0].to(d) * s["x"].to(d)
    for j in range(1, T):
        p = p + s["w"][:, j].to(d) * s["state"][:, :, T - 1 - j].to(d)
    y = p / (1 + torch.exp(-p)) if c["silu"] else p
    return y, torch.cat((s["state"][:, :, 1:], s["x"][:, :, None]), 2).to(d)[:, :, :T - 1]


def _exact_scan(s, c):
    """The recurrence, one step after the other."""
    d = torch.float64
    B, D, L, N, G = c["B"], c["D"], c.get("L", 1), c["N"], c["G"]
    single, back = c["op"] == "scan_step", c["op"] == "scan_bwd"
    along = lambda v: v.unsqueeze(-1) if single else v  # noqa: E731
    n = s["lengths"].tolist() if s.get("lengths") is not None else [L] * B
    u, delta, Bm, Cm = (torch.zeros(v.shape, dtype=d, device=DEV) for v in map(along, (s["u"], s["delta"], s["Bm"], s["Cm"])))
    z, gy = torch.zeros_like(u), torch.zeros_like(u)
    dt, sig = torch.zeros_like(u), torch.zeros_like(u)
    for b, m in enumerate(n):
        u[b, :, :m], delta[b, :, :m] = along(s["u"])[b, :, :m].to(d), along(s["delta"])[b, :, :m].to(d)
        Bm[b, :, :, :m], Cm[b, :, :, :m] = along(s["Bm"])[b, :, :, :m].to(d), along(s["Cm"])[b, :, :, :m].to(d)
        x = delta[b, :, :m] + s["delta_bias"].to(d)[:, None]
        dt[b, :, :m] = torch.logaddexp(x, torch.zeros_like(x))
        sig[b, :, :m] = 1 / (1 + torch.exp(-x))
        if s["z"] is not None:
            z[b, :, :m] = along(s["z"])[b, :, :m].to(d)
        if back:
            gy[b, :, :m] = s["gy"][b, :, :m].to(d)
    A, skip = s["A"].to(d), s["skip"].to(d)[:, None]
    h = s["state"].to(d) if s["state"] is not None else torch.zeros(B, D, N, dtype=d, device=DEV)
    first = h
    at = lambda v, t: v[..., t].unsqueeze(2).expand(B, G, D // G, N).reshape(B, D, N)  # noqa: E731
    y = torch.empty_like(u)
    kept = torch.empty(L if back else 0, B, D, N, dtype=d, device=DEV)
    for t in range(L):
        h = torch.exp(dt[:, :, t, None] * A) * h + (dt[:, :, t] * u[:, :, t])[..., None] * at(Bm, t)
        y[:, :, t] = (h * at(Cm, t)).sum(-1)
        if back:
            kept[t] = h
    y += skip * u
    gate = z / (1 + torch.exp(-z)) if s["z"] is not None else torch.ones_like(u)
    if not back:
        y = y * gate
        return (y[..., 0] if single else y), h
    gz = None
    if s["z"] is not None:
        sz = 1 / (1 + torch.exp(-z))
        gz = gy * y * (sz + z * sz * (1 - sz))
    gy = gy * gate
    gB, gC, gu, gdt = torch.zeros_like(Bm), torch.zeros_like(Cm), torch.empty_like(u), torch.empty_like(u)
    gA = torch.zeros_like(A)
    gh = s["gstate_out"].to(d) if s["gstate_out"] is not None else torch.zeros_like(h)
    for t in range(L - 1, -1, -1):
        gh = gh + gy[:, :, t, None] * at(Cm, t)
        gC[..., t] = (kept[t] * gy[:, :, t, None]).reshape(B, G, D // G, N).sum(2)
        gB[..., t] = (gh * (dt[:, :, t] * u[:, :, t])[..., None]).reshape(B, G, D // G, N).sum(2)
        gb = (gh * at(Bm, t)).sum(-1)
        gh = gh * torch.exp(dt[:, :, t, None] * A)  # now with respect to h[t-1]
        w = gh * (kept[t - 1] if t else first)
        gA += (w * dt[:, :, t, None]).sum(0)
        gdt[:, :, t] = (w * A).sum(-1) + gb * u[:, :, t]
        gu[:, :, t] = gb * dt[:, :, t]
    gdelta = gdt * sig
    return {"gu": gu + skip * gy, "gdelta": gdelta, "gA": gA, "gB": gB, "gC": gC, "gskip": (gy * u).sum((0, 2)), "gz": gz,
            "gdelta_bias": gdelta.sum((0, 2)), "gstate": gh if s["state"] is not None else None}


def _exact_quantized(v, rows):
    """The values that the 8-bit codes of v [R, K] stand for, and the scales, which are held in 32 bits by definition."""
    R, K = v.shape
    scales = torch.zeros(-(-R // rows), -(-K // 128), dtype=torch.float64, device=DEV)
    held = torch.empty_like(v)
    for k in range(scales.shape[1]):
        part = v[:, 128 * k:128 * k + 128]
        top = part.abs().amax(1)
        top = torch.nn.functional.pad(top, (0, -R % rows)).view(-1, rows).amax(1)
        scales[:, k] = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top)).float().double()
        each = scales[:, k].repeat_interleave(rows)[:R, None]
        held[:, 128 * k:128 * k + 128] = (part / each).float().to(torch.float8_e4m3fn).double() * each
    return held, scales


def _exact_norm(s, c):
    d = torch.float64
    v = s["x"].to(d)
    if c["op"] == "norm_bwd":
        gy, w = s["gy"].to(d), s["weight"].to(d)
        ms = v.square().sum(-1, keepdim=True) / c["D"] + EPS
        gx = gy * w / ms.sqrt() - v * (gy * w * v).sum(-1, keepdim=True) / (c["D"] * ms * ms.sqrt())
        if s["gs"] is not None:
            gx = gx + s["gs"].to(d)
        return gx, (gy * v / ms.sqrt()).sum(0)
    carried = ()
    if s["residual"] is not None:
        v = (v + s["residual"].to(d)).to(s["x"].dtype).to(d)  # the sum is stored, and its stored value is normed
        carried = (v,)
    y = v / (v.square().sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * s["weight"].to(d)
    if c["op"] == "norm":
        return (y, *carried)
    held, scales = _exact_quantized(y, 1)
    return (held, scales, *carried)


def _exact_product(s, c):
    d = torch.float64
    left = s["q"].to(d) * _spread(s["scales"].to(d), c["M"], c["K"], 1) if "q" in s else _exact_quantized(s["x"].to(d), 1)[0]
    right = s["wq"].to(d) * _spread(s["wscales"].to(d), c["N"], c["K"], 128)
    out = torch.mm(right, left.t().contiguous())
    if s["bias"] is not None:
        out = out + s["bias"].to(d)[:, None]
    return out if c["channel_major"] else out.t().contiguous()


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "conv_step":
        return _exact_conv_step(s, c)
    if c["op"].startswith("conv"):
        return _exact_conv(s, c)
    if c["op"].startswith("scan"):
        return _exact_scan(s, c)
    if c["op"].startswith("norm"):
        return _exact_norm(s, c)
    return _exact_product(s, c)
