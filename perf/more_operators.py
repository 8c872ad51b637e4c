"""Measured cases of the linear-attention block's operators.

The block: rotary positions on queries and keys, linear attention with a decay
for each head, and a norm of each head's outputs with a gate.  Activations are
token-major, [B, L, heads, head size], as a row-major projection leaves them.

    linear attention    S[t] = exp(log_decay) S[t-1] + k[t] v[t]^T,  o[t] = scale S[t]^T q[t]
    rotary positions    (a, b) -> scale (a cos - b sin, a sin + b cos),  angle = position * frequency
    group norm          n = (x - mean) / sqrt(var + eps) over a row's group,  m = n weight + bias,
                        y = m, m * sigmoid(m), or m * z * sigmoid(z)

`run` computes the plain forms with elementary torch operations, or, where
`own` is set, calls this package.  `exact` is the same in float64.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
CHUNK = 64  # tokens of a block in the plain form


def listed():
    return [
        # Linear attention in a training step's forward pass.
        dict(name="attn_training", op="attn", dtype="bf16", B=8, L=2048, H=12, Hq=12, Hk=12, Hv=12, Dk=64, Dv=128, state=False, lengths=False,
             decay=True, fused=False),
        # Ragged, right-padded prompts of an odd length; q, k and v are parts of one projection's rows, k and v shared by three heads.
        dict(name="attn_prompts", op="attn", dtype="bf16", B=5, L=3001, H=12, Hq=12, Hk=4, Hv=4, Dk=64, Dv=64, state=False, lengths=True,
             decay=True, fused=True),
        # One long sequence (the 64K-token shape): few heads, so the time axis has to be split.
        dict(name="attn_long", op="attn", dtype="bf16", B=1, L=65536, H=6, Hq=6, Hk=6, Hv=6, Dk=128, Dv=128, state=True, lengths=False,
             decay=True, fused=False),
        # The same length in fp32.
        dict(name="attn_long_fp32", op="attn", dtype="fp32", B=1, L=65536, H=12, Hq=12, Hk=12, Hv=12, Dk=64, Dv=64, state=False, lengths=False,
             decay=True, fused=False),
        # The gradients in a training step.
        dict(name="attn_backward", op="attn_bwd", dtype="bf16", B=4, L=2048, H=12, Hq=12, Hk=12, Hv=12, Dk=64, Dv=128, state=False,
             lengths=False, decay=True, fused=False),
        # One new token for each of 128 sequences: the states' traffic.
        dict(name="attn_token", op="attn_step", dtype="bf16", B=128, H=12, Hq=12, Hk=12, Hv=12, Dk=64, Dv=128, decay=True, fused=False),
        # One new token for each of 4 sequences: latency.
        dict(name="attn_token_few", op="attn_step", dtype="bf16", B=4, H=12, Hq=12, Hk=4, Hv=4, Dk=64, Dv=64, decay=True, fused=True),
        # The norm of the heads' outputs with a gate, activations of a training step.
        dict(name="norm_gated", op="gnorm", dtype="bf16", rows=16384, G=12, Dg=128, act="gate", affine=True),
        # Its gradients.
        dict(name="norm_backward", op="gnorm_bwd", dtype="bf16", rows=16384, G=12, Dg=128, act="gate", affine=True),
        # Rotary positions on the queries and keys of a batch of prompts.
        dict(name="rotary_prompts", op="rotary", dtype="bf16", B=8, L=2048, H=24, D=64, R=64, interleaved=False, inverse=False, far=False,
             scaling="none"),
        # Half of each head turned, at far positions of a context that was stretched, in fp32.
        dict(name="rotary_far", op="rotary", dtype="fp32", B=1, L=65536, H=12, D=64, R=32, interleaved=False, inverse=False, far=True,
             scaling="yarn"),
        # One new token for each of 16 sequences, interleaved pairs: the smallest call, all latency.
        dict(name="rotary_token", op="rotary", dtype="bf16", B=16, L=1, H=24, D=64, R=64, interleaved=True, inverse=False, far=True,
             scaling="none"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    """H, and the heads of q, k and v: all alike, k and v shared by several heads, or q and k shared."""
    H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    few = rng.choice([d for d in range(1, H + 1) if H % d == 0])
    Hq, Hk, Hv = rng.choice([(H, H, H), (H, H, H), (H, few, few), (few, few, H)])
    return dict(H=H, Hq=Hq, Hk=Hk, Hv=Hv)


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn_bwd", "attn_bwd", "attn_step", "gnorm", "gnorm_bwd", "rotary", "rotary"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp32"]))
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("attn"):
        c.update(_heads(rng), Dk=rng.choice([16, 32, 40, 64, 64, 96, 128, 128, 256]), Dv=rng.choice([16, 32, 64, 64, 80, 128, 128, 200, 256]),
                 decay=rng.random() < 0.8, fused=yes())
        each = c["H"] * c["Dk"] * c["Dv"]
        if op == "attn_step":
            c["B"] = max(1, min(_log(rng, 1, 256), 12_000_000 // each))
            return c
        most = 6_000_000_000 if op == "attn" else 2_000_000_000
        B, L = _log(rng, 1, 16), _log(rng, 1, 65536 if op == "attn" else 32768)
        L = max(1, min(L, most // (B * each), 100_000_000 // (B * c["H"] * (c["Dk"] + c["Dv"]))))
        c.update(B=B, L=L, state=yes(), lengths=yes())
    elif op.startswith("gnorm"):
        G, Dg = rng.choice([1, 2, 4, 8, 12, 16, 24, 32]), _log(rng, 8, 2048)
        c.update(rows=max(1, min(_log(rng, 1, 65536), 25_000_000 // (G * Dg))), G=G, Dg=Dg, act=rng.choice(["none", "silu", "gate", "gate"]),
                 affine=yes())
    else:
        H, D = _log(rng, 1, 32), rng.choice([32, 48, 64, 64, 80, 96, 128, 128, 256])
        B, L = _log(rng, 1, 64), _log(rng, 1, 65536)
        c.update(B=B, L=max(1, min(L, 25_000_000 // (B * H * D))), H=H, D=D, R=rng.choice([D, D, D // 2, D // 4 * 2]), interleaved=yes(),
                 inverse=yes(), far=yes(), scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
    return c


# ------------------------------------------------------------------ inputs

def _attn_inputs(c, r, u, t):
    B, H, Dk, Dv = c["B"], c["H"], c["Dk"], c["Dv"]
    lead = (B,) if c["op"] == "attn_step" else (B, c["L"])
    widths = (c["Hq"] * Dk, c["Hk"] * Dk, c["Hv"] * Dv)
    if c["fused"]:  # parts of one projection's rows
        q, k, v = r(*lead, sum(widths)).to(t).split(widths, -1)
    else:
        q, k, v = (r(*lead, n).to(t) for n in widths)
    s = {"q": q.unflatten(-1, (c["Hq"], Dk)), "k": k.unflatten(-1, (c["Hk"], Dk)), "v": v.unflatten(-1, (c["Hv"], Dv)),
         # from heads that remember thousands of tokens to those that remember a few
         "log_decay": -torch.exp(math.log(1e-4) + u(H) * math.log(1e4)) if c["decay"] else None}
    if c["op"] == "attn_step" or c["state"]:
        s["state"] = r(B, H, Dk, Dv)
    else:
        s["state"] = None
    if c["op"] == "attn_bwd":
        s.update(go=r(*lead, H, Dv).to(t), gstate_out=r(B, H, Dk, Dv) if c["state"] else None)
    if c["op"] != "attn_step":
        s["lengths"] = None
        if c["lengths"]:  # right-padded prompts: the padding holds whatever was there
            n = (u(B) * (c["L"] + 1)).to(torch.int32).clamp_(max=c["L"])
            n[0] = c["L"]
            s["lengths"] = n
    return s


def _frequencies(c):
    """The angle of one position for each pair, float64 [R/2], and the factor of the outputs."""
    R, base, stretch, first = c["R"], 10000.0, 8.0, 4096.0
    i = torch.arange(0, R, 2, dtype=torch.float64) / R
    f = base ** -i
    if c["scaling"] == "linear":
        return f / stretch, 1.0
    if c["scaling"] == "ntk":
        return (base * stretch ** (R / (R - 2))) ** -i, 1.0
    if c["scaling"] == "yarn":  # pairs that turn often within the first context keep their frequency, slow ones are stretched
        keep = ((first * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * keep + f / stretch * (1 - keep), 0.1 * math.log(stretch) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *n: torch.randn(*n, generator=g, device=DEV)  # noqa: E731
    u = lambda *n: torch.rand(*n, generator=g, device=DEV)  # noqa: E731
    c, t = case, TYPES[case["dtype"]]
    op = c["op"]
    if op.startswith("attn"):
        s = _attn_inputs(c, r, u, t)
    elif op.startswith("gnorm"):
        rows, D = c["rows"], c["G"] * c["Dg"]
        s = {"x": (2 * r(rows, D) + 0.5 * r(rows, 1)).to(t), "z": r(rows, D).to(t) if c["act"] == "gate" else None,
             "weight": 1 + 0.2 * r(D) if c["affine"] else None, "bias": 0.2 * r(D) if c["affine"] else None}
        if op == "gnorm_bwd":
            s["gy"] = r(rows, D).to(t)
    else:
        freq, scale = _frequencies(c)
        s = {"x": r(c["B"], c["L"], c["H"], c["D"]).to(t), "freq": freq.to(DEV), "scale": scale, "positions": None}
        if c["far"]:  # each sequence goes on from a place of its own
            start = (u(c["B"], 1) * (1 << 20)).to(torch.int32)
            s["positions"] = start + torch.arange(c["L"], device=DEV, dtype=torch.int32)
    s["case"] = c
    return s


# ------------------------------------------------------------- plain forms

def _chunks(s, c):
    """q, k, v (and go) in blocks [B, H, n, CHUNK, D] of 32-bit values, zeros behind a length, with what the decays need: the tokens of each
    block that count, and powers of a head's decay."""
    B, L, H = c["B"], c["L"], c["H"]
    n = -(-L // CHUNK)
    at = torch.arange(n * CHUNK, device=DEV)
    length = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), L, device=DEV)

    def blocks(x):
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, n * CHUNK - L))
        x = torch.where((at < length[:, None])[:, :, None, None], x, torch.zeros((), device=DEV))
        x = x.repeat_interleave(H // x.shape[2], 2)
        return x.reshape(B, n, CHUNK, H, -1).permute(0, 3, 1, 2, 4).contiguous()

    g = s["log_decay"] if s["log_decay"] is not None else torch.zeros(H, device=DEV)
    m = (length[:, None] - CHUNK * torch.arange(n, device=DEV)).clamp(0, CHUNK)  # [B, n]
    e = torch.minimum(torch.arange(1, CHUNK + 1, device=DEV), m[..., None])  # decays from the block's start through token i
    power = lambda p: torch.exp(g.view(1, H, *[1] * (p.dim() - 1)) * p[:, None])  # noqa: E731
    within = torch.where(torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril(), power(e[..., :, None] - e[..., None, :]),
                         torch.zeros((), device=DEV))
    return blocks, within, power(e)[..., None], power(m[..., None] - e)[..., None], power(m)[..., None, None]


def _prefix(a, b):
    """h[i] = a[i] h[i-1] + b[i] along the third axis, by pairs."""
    n = b.shape[2]
    if n == 1:
        return b
    m = n // 2 * 2
    odd = _prefix(a[:, :, 1:m:2] * a[:, :, 0:m:2], a[:, :, 1:m:2] * b[:, :, 0:m:2] + b[:, :, 1:m:2])
    h = torch.empty_like(b)
    h[:, :, 0] = b[:, :, 0]
    h[:, :, 1:m:2] = odd
    h[:, :, 2::2] = a[:, :, 2::2] * odd[:, :, :(n - 1) // 2] + b[:, :, 2::2]
    return h


def _carry(first, local, decay):
    """The states before each block, and the one that is left."""
    local[:, :, 0] += decay[:, :, 0] * first
    h = _prefix(decay, local)
    return torch.cat((first[:, :, None], h[:, :, :-1]), 2), h[:, :, -1].contiguous()


def _as_tokens(x, L):
    B, H, n, C, D = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, D)[:, :L]


def _zeros_state(s, c, key):
    return s[key] if s[key] is not None else torch.zeros(c["B"], c["H"], c["Dk"], c["Dv"], device=DEV)


def _attn(s, c):
    blocks, within, through, left, whole = _chunks(s, c)
    q, k, v = blocks(s["q"]) * c["Dk"] ** -0.5, blocks(s["k"]), blocks(s["v"])
    before, last = _carry(_zeros_state(s, c, "state"), (k * left).transpose(-1, -2) @ v, whole)
    o = (q @ k.transpose(-1, -2) * within) @ v + (q * through) @ before
    return _as_tokens(o, c["L"]).to(s["q"].dtype).contiguous(), last


def _attn_bwd(s, c):
    blocks, within, through, left, whole = _chunks(s, c)
    scale, t, L = c["Dk"] ** -0.5, s["q"].dtype, c["L"]
    q, k, v, go = blocks(s["q"]) * scale, blocks(s["k"]), blocks(s["v"]), blocks(s["go"])
    before, _ = _carry(_zeros_state(s, c, "state"), (k * left).transpose(-1, -2) @ v, whole)
    behind, first = _carry(_zeros_state(s, c, "gstate_out"), ((q * through).transpose(-1, -2) @ go).flip(2), whole.flip(2))
    behind = behind.flip(2)
    P, dP = q @ k.transpose(-1, -2) * within, go @ v.transpose(-1, -2) * within
    gq = (dP @ k + (go * through) @ before.transpose(-1, -2)) * scale
    gk = dP.transpose(-1, -2) @ q + (v * left) @ behind.transpose(-1, -2)
    gv = P.transpose(-1, -2) @ go + (k * left) @ behind
    fold = lambda x, heads: _as_tokens(x, L).unflatten(2, (heads, -1)).sum(3).to(t)  # noqa: E731: over the heads that share it
    return {"gq": fold(gq, c["Hq"]), "gk": fold(gk, c["Hk"]), "gv": fold(gv, c["Hv"]), "gstate": first if s["state"] is not None else None}


def _attn_step(s, c):
    H = c["H"]
    wide = lambda x: x.float().repeat_interleave(H // x.shape[1], 1)  # noqa: E731
    q, k, v = wide(s["q"]) * c["Dk"] ** -0.5, wide(s["k"]), wide(s["v"])
    kv = k[..., :, None] * v[..., None, :]
    new = s["state"] * torch.exp(s["log_decay"])[:, None, None] + kv if s["log_decay"] is not None else s["state"] + kv
    s["state"].copy_(new)
    return (q[..., :, None] * new).sum(-2).to(s["q"].dtype), s["state"]


def _gnorm_parts(s, c):
    x = s["x"].float().unflatten(-1, (c["G"], c["Dg"]))
    d = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    n = (d * rstd).flatten(-2)
    m = n * s["weight"] + s["bias"] if c["affine"] else n
    return rstd, n, m


def _gnorm(s, c):
    _, _, m = _gnorm_parts(s, c)
    if c["act"] == "silu":
        m = m * torch.sigmoid(m)
    elif c["act"] == "gate":
        z = s["z"].float()
        m = m * z * torch.sigmoid(z)
    return m.to(s["x"].dtype)


def _gnorm_bwd(s, c):
    t = s["x"].dtype
    rstd, n, m = _gnorm_parts(s, c)
    gm, gz = s["gy"].float(), None
    if c["act"] == "silu":
        sig = torch.sigmoid(m)
        gm = gm * sig * (1 + m * (1 - sig))
    elif c["act"] == "gate":
        z = s["z"].float()
        sig = torch.sigmoid(z)
        gz = (gm * m * sig * (1 + z * (1 - sig))).to(t)
        gm = gm * z * sig
    split = lambda v: v.unflatten(-1, (c["G"], c["Dg"]))  # noqa: E731
    gn, n3 = split(gm * s["weight"] if c["affine"] else gm), split(n)
    gx = rstd * (gn - gn.mean(-1, keepdim=True) - n3 * (gn * n3).mean(-1, keepdim=True))
    return {"gx": gx.flatten(-2).to(t), "gweight": (gm * n).sum(0, dtype=torch.float64).float() if c["affine"] else None,
            "gbias": gm.sum(0, dtype=torch.float64).float() if c["affine"] else None, "gz": gz}


def _rotary(s, c):
    R, x = c["R"], s["x"]
    at = s["positions"] if s["positions"] is not None else torch.arange(c["L"], device=DEV)[None]
    angle = (at.double()[..., None] * s["freq"])[:, :, None]  # [B, L, 1, R/2]
    cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    if c["inverse"]:
        sin = -sin
    v = x[..., :R].float()
    if c["interleaved"]:
        a, b = v[..., 0::2], v[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = v[..., :R // 2], v[..., R // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned.to(x.dtype), x[..., R:]), -1)


PLAIN = {"attn": _attn, "attn_bwd": _attn_bwd, "attn_step": _attn_step, "gnorm": _gnorm, "gnorm_bwd": _gnorm_bwd, "rotary": _rotary}


# ---------------------------------------------------------- this package's

def _run_own(s, c):
    import hyena_long_conv_amd as H
    op = c["op"]
    if op == "attn":
        return H.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], lengths=s["lengths"], return_state=True)
    if op == "attn_bwd":
        return H.linear_attention_backward(s["q"], s["k"], s["v"], s["go"], s["log_decay"], state=s["state"], lengths=s["lengths"],
                                           gstate_out=s["gstate_out"])
    if op == "attn_step":
        return H.linear_attention_step(s["q"], s["k"], s["v"], s["state"], s["log_decay"]), s["state"]
    if op == "gnorm":
        return H.group_norm(s["x"], c["G"], s["weight"], s["bias"], z=s["z"], silu=c["act"] == "silu", eps=EPS)
    if op == "gnorm_bwd":
        return H.group_norm_backward(s["x"], c["G"], s["gy"], s["weight"], s["bias"], z=s["z"], silu=c["act"] == "silu", eps=EPS)
    return H.rotary(s["x"], s["freq"], s["positions"], scale=s["scale"], interleaved=c["interleaved"], inverse=c["inverse"])


def run(state):
    c = state["case"]
    return _run_own(state, c) if own else PLAIN[c["op"]](state, c)


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    op = c["op"]
    if op.startswith("attn"):
        tokens, Dk, Dv = c["B"] * c.get("L", 1), c["Dk"], c["Dv"]
        read = e * tokens * ((c["Hq"] + c["Hk"]) * Dk + c["Hv"] * Dv)
        o, states, each = e * tokens * c["H"] * Dv, 4 * c["B"] * c["H"] * Dk * Dv, tokens * c["H"] * Dk * Dv
        if op == "attn_step":
            return {"bytes": read + o + 2 * states, "flops": 5 * each}
        if op == "attn":
            return {"bytes": read + o + states * (2 if c["state"] else 1), "flops": 4 * each}
        return {"bytes": 2 * read + o + states * (3 if c["state"] else 0), "flops": 10 * each}
    if op.startswith("gnorm"):
        n, gate, rest = c["rows"] * c["G"] * c["Dg"], c["act"] == "gate", 8 * c["G"] * c["Dg"] * c["affine"]
        if op == "gnorm":
            return {"bytes": e * n * (3 if gate else 2) + rest, "flops": n * (12 if c["act"] != "none" else 7)}
        return {"bytes": e * n * (5 if gate else 3) + 2 * rest, "flops": n * (26 if c["act"] != "none" else 16)}
    n, tokens = c["B"] * c["L"] * c["H"], c["B"] * c["L"]
    return {"bytes": 2 * e * n * c["D"] + (4 * tokens if c["far"] else 0) + 4 * c["R"], "flops": 3 * n * c["R"] + 20 * tokens * c["R"]}


# ---------------------------------------------------------------- 64 bits

def _exact_attn(s, c):
    """The recurrence, one token after the other; its gradients by the same recurrence forward and backward in time."""
    d, single, back = torch.float64, c["op"] == "attn_step", c["op"] == "attn_bwd"
    B, L, H, Dk, Dv = c["B"], c.get("L", 1), c["H"], c["Dk"], c["Dv"]
    n = s["lengths"] if s.get("lengths") is not None else torch.full((B,), L, device=DEV)
    inside = (torch.arange(L, device=DEV)[:, None] < n[None])  # [L, B]

    def first(x):  # time in front, every head its own copy
        x = x[:, None] if single else x
        x = torch.where(inside.t()[:, :, None, None], x, torch.zeros((), dtype=x.dtype, device=DEV))
        return x.transpose(0, 1).to(d).repeat_interleave(H // x.shape[2], 2).contiguous()

    q, k, v = first(s["q"]), first(s["k"]), first(s["v"])
    lam = torch.exp(s["log_decay"].to(d)) if s["log_decay"] is not None else torch.ones(H, dtype=d, device=DEV)
    step = torch.where(inside[..., None], lam, torch.ones((), dtype=d, device=DEV))[..., None, None]  # [L, B, H, 1, 1]
    scale = Dk ** -0.5
    S = s["state"].to(d) if s["state"] is not None else torch.zeros(B, H, Dk, Dv, dtype=d, device=DEV)
    left = torch.empty(L, B, H, Dk if back else Dv, dtype=d, device=DEV)  # o, or gq
    go = first(s["go"]) if back else None
    S = S.clone()
    for t in range(L):
        S.mul_(step[t]).addcmul_(k[t][..., :, None], v[t][..., None, :])
        left[t] = (S * go[t][..., None, :]).sum(-1) if back else (S * q[t][..., :, None]).sum(-2)
    left = scale * left
    if single:
        return left[0], S
    tokens = lambda x: x.transpose(0, 1)  # noqa: E731
    if not back:
        return tokens(left), S
    G = s["gstate_out"].to(d).clone() if s["gstate_out"] is not None else torch.zeros_like(S)
    gk, gv = torch.empty_like(k), torch.empty_like(v)
    q = scale * q
    for t in range(L - 1, -1, -1):
        G.addcmul_(q[t][..., :, None], go[t][..., None, :])
        gk[t] = (G * v[t][..., None, :]).sum(-1)
        gv[t] = (G * k[t][..., :, None]).sum(-2)
        G.mul_(step[t])
    fold = lambda x, heads: tokens(x).reshape(B, L, heads, H // heads, -1).sum(3)  # noqa: E731
    return {"gq": fold(left, c["Hq"]), "gk": fold(gk, c["Hk"]), "gv": fold(gv, c["Hv"]), "gstate": G if s["state"] is not None else None}


def _exact_gnorm(s, c):
    d = torch.float64
    x = s["x"].to(d).view(c["rows"], c["G"], c["Dg"])
    D = c["G"] * c["Dg"]
    w = s["weight"].to(d) if c["affine"] else torch.ones(D, dtype=d, device=DEV)
    b = s["bias"].to(d) if c["affine"] else torch.zeros(D, dtype=d, device=DEV)
    mean = x.sum(-1, keepdim=True) / c["Dg"]
    std = (((x - mean) ** 2).sum(-1, keepdim=True) / c["Dg"] + EPS).sqrt()
    n = (x - mean) / std
    m = n.view(c["rows"], D) * w + b
    z = s["z"].to(d) if c["act"] == "gate" else m
    slope = None
    if c["act"] != "none":
        sz = 1 / (1 + torch.exp(-z))
        slope = sz + z * sz * (1 - sz)
    if c["op"] == "gnorm":
        return m if c["act"] == "none" else z * sz if c["act"] == "silu" else m * z * sz
    gy = s["gy"].to(d)
    gm = gy if c["act"] == "none" else gy * slope if c["act"] == "silu" else gy * z * sz
    gz = gy * m * slope if c["act"] == "gate" else None
    gn = (gm * w).view_as(n)
    gx = (gn - gn.sum(-1, keepdim=True) / c["Dg"] - n * (gn * n).sum(-1, keepdim=True) / c["Dg"]) / std
    return {"gx": gx.view(c["rows"], D), "gweight": (gm * n.view(c["rows"], D)).sum(0) if c["affine"] else None,
            "gbias": gm.sum(0) if c["affine"] else None, "gz": gz}


def _exact_rotary(s, c):
    d, R = torch.float64, c["R"]
    x = s["x"].to(d)
    at = s["positions"].to(d) if s["positions"] is not None else torch.arange(c["L"], dtype=d, device=DEV).expand(c["B"], -1)
    out = x.clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
        angle = at * s["freq"][i] * (-1 if c["inverse"] else 1)
        turn = torch.polar(torch.full_like(angle, s["scale"]), angle)[:, :, None]  # scale e^(i angle)
        pair = torch.complex(x[..., a], x[..., b]) * turn
        out[..., a], out[..., b] = pair.real, pair.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("attn"):
        return _exact_attn(s, case)
    return _exact_gnorm(s, case) if case["op"].startswith("gnorm") else _exact_rotary(s, case)
