"""The linear-attention block's operators on the GPU against their float64
definitions (tests/linattn_reference.py), values and gradients, at the sizes
and masks where tiles, words and segments end.

Tolerances.  With half the I/O dtype's half step (2^-8 bf16, 2^-24 fp32) and
size the sum of the sizes of a value's terms, an output is compared within

    half * |ref| + (r * half + c * 2^-24) * size:

one rounding where the value is stored, r roundings of a term to the I/O dtype
on the way (bf16 attention: the weight of a pair of tokens inside a block, or
the state in front of it: r = 1; none elsewhere), and c fp32 roundings of a
term.  c is counted at each test."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests import linattn_reference as R
from tests import ssm_reference as S
from tests.test_ssm import DEV, EPS32, HALF, TYPES, dev, gen, leaves

pytestmark = pytest.mark.gpu


def near(got, ref, size, c, r=0, what=""):
    got64, ref, size = got.detach().cpu().double(), ref.detach().cpu(), size.cpu() if isinstance(size, torch.Tensor) else size
    assert got64.shape == ref.shape, (what, got64.shape, ref.shape)
    assert bool(torch.isfinite(got64).all()), f"{what}: not finite"
    if ref.numel():
        half = HALF[got.dtype]
        off = (got64 - ref).abs() / (half * ref.abs() + (r * half + c * EPS32) * size + 1e-37)
        assert float(off.max()) <= 1, f"{what}: {float(off.max()):.3g} times its tolerance"


# ---------------------------------------------------------- linear attention

def count(L, Dk, Dv):
    """fp32 roundings of a term: a dot product of Dk or Dv, sums over a block of 64 tokens and over the blocks, each with a
    decay; 32 for the decays' exponentials, the scale, and the states joined between segments."""
    return max(Dk, Dv) + 64 + 2 * (L / 32) + 32


def attention_inputs(case, t, seed):
    B, L, heads, Dk, Dv, has_state, lens, decay, layout = case
    r = gen(seed)
    Hq, Hk, Hv = heads
    N = max(heads)
    if layout == "fused":                               # parts of one projection's rows
        q, k, v = r(B, L, Hq * Dk + Hk * Dk + Hv * Dv).to(t).split((Hq * Dk, Hk * Dk, Hv * Dv), -1)
        q, k, v = q.unflatten(-1, (Hq, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (Hv, Dv))
    elif layout == "heads first":
        q, k, v = (r(B, h, L, d).to(t).transpose(1, 2) for h, d in ((Hq, Dk), (Hk, Dk), (Hv, Dv)))
    else:
        q, k, v = (r(B, L, h, d).to(t) for h, d in ((Hq, Dk), (Hk, Dk), (Hv, Dv)))
    g = {"none": None, "zero": torch.zeros(N), "fast": -3 * torch.rand(N, generator=torch.Generator().manual_seed(seed)),
         "slow": -torch.exp(-2 - 6 * torch.rand(N, generator=torch.Generator().manual_seed(seed))),
         "off": torch.full((N,), float("-inf"))}[decay]
    a = dict(q=q, k=k, v=v, log_decay=g, state=r(B, N, Dk, Dv) if has_state else None,
             lengths=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    return a, r(B, L, N, Dv).to(t), r(B, N, Dk, Dv) if has_state else None


def spoil(t, lengths):
    """NaN and infinities behind each sequence's length (time is the second axis), in t's own layout."""
    if lengths is None:
        return t
    for b, n in enumerate(S.clamp_lengths(lengths, t.shape[0], t.shape[1])):
        t[b, n:] = float("nan")
        if n < t.shape[1]:
            t[b, -1] = float("inf")
    return t


def on_gpu(a):
    """Arguments on the GPU with their strides, what lies behind a length spoilt."""
    out = {}
    for k, t in a.items():
        if t is None:
            out[k] = None
        elif k in ("q", "k", "v") and not t.is_contiguous():
            base = t._base if t._base is not None else t
            out[k] = torch.as_strided(base.to(DEV), t.shape, t.stride(), t.storage_offset())
        else:
            out[k] = t.to(DEV)
        if k in ("q", "k", "v"):
            spoil(out[k], a["lengths"])
    return out


ATTENTION = [
    # B, L, heads of q k v, Dk, Dv, state, lengths, decay, layout
    (1, 1, (1, 1, 1), 1, 1, False, None, "slow", "dense"),
    (2, 1, (3, 3, 3), 16, 8, True, None, "slow", "dense"),
    (2, 2, (2, 2, 2), 3, 5, True, [0, 2], "fast", "dense"),
    (1, 15, (2, 2, 2), 32, 32, False, None, "none", "dense"),
    (2, 17, (2, 1, 1), 40, 24, True, [17, 3], "slow", "fused"),
    (3, 31, (1, 1, 2), 64, 64, True, [-4, 31, 100], "slow", "dense"),
    (2, 33, (4, 2, 1), 64, 128, False, None, "fast", "heads first"),
    (1, 63, (2, 2, 2), 65, 65, True, None, "slow", "dense"),
    (2, 64, (1, 2, 1), 64, 64, True, None, "zero", "fused"),
    (2, 65, (2, 2, 2), 128, 128, True, [65, 64], "slow", "dense"),
    (2, 100, (2, 2, 2), 96, 80, True, [1, 99], "off", "dense"),
    (1, 127, (2, 2, 1), 33, 129, True, None, "slow", "fused"),
    (1, 129, (1, 1, 1), 256, 256, True, None, "slow", "dense"),
    (2, 130, (2, 1, 2), 200, 17, False, [129, 128], "fast", "dense"),
    (2, 193, (3, 3, 1), 17, 250, True, [64, 193], "slow", "heads first"),
    (1, 321, (2, 2, 2), 128, 64, True, None, "slow", "dense"),
    (2, 300, (2, 2, 2), 1, 256, True, [300, 0], "slow", "dense"),
    (1, 300, (2, 2, 2), 256, 1, True, None, "slow", "dense"),
]


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("case", ATTENTION, ids=str)
def test_linear_attention(case, io):
    t = TYPES[io]
    B, L, _, Dk, Dv = case[:5]
    a, go, gso = attention_inputs(case, t, L + Dk)
    ref = R.linear_attention(**a, go=go, gstate_out=gso)
    on = on_gpu(a)
    o, last = H.linear_attention(**on, return_state=True)
    c, r = count(L, Dk, Dv), 1 if io == "bf16" else 0
    near(o, *ref["o"], c, r, "o")
    near(last, *ref["state"], c, 0, "state")
    assert torch.equal(H.linear_attention(**on), o), "the same without the state"
    got = H.linear_attention_backward(**on, go=spoil(go.to(DEV), a["lengths"]), gstate_out=dev(gso))
    for name in ("gq", "gk", "gv"):
        near(got[name], *ref[name], c + 8, r, name)
    assert (got["gstate"] is None) == (a["state"] is None)
    if gso is not None:
        near(got["gstate"], *ref["gstate"], c, 0, "gstate")
    if a["lengths"] is not None:
        for b, n in enumerate(S.clamp_lengths(a["lengths"], B, L)):
            for name, x in [("o", o), *got.items()]:
                if name != "gstate":
                    assert not bool(x[b, n:].any()), f"{name} behind a length"


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("B,heads,Dk,Dv,decay", [(1, (1, 1, 1), 1, 1, "slow"), (3, (4, 2, 2), 64, 64, "slow"), (2, (2, 2, 4), 128, 100, "fast"),
                                                 (2, (1, 3, 3), 40, 33, "none"), (2, (2, 2, 2), 256, 256, "zero"), (5, (2, 2, 2), 7, 250, "off"),
                                                 (300, (1, 1, 1), 16, 8, "slow")])
def test_linear_attention_step(B, heads, Dk, Dv, decay, io):
    """Tokens one at a time leave what a prompt of them does."""
    t, L = TYPES[io], 3
    a, _, _ = attention_inputs((B, L, heads, Dk, Dv, True, None, decay, "fused"), t, B + Dk)
    ref = R.linear_attention(**a)
    on = on_gpu(a)
    state = on.pop("state")
    on.pop("lengths")
    for i in range(L):
        o = H.linear_attention_step(on["q"][:, i], on["k"][:, i], on["v"][:, i], state, on["log_decay"])
        near(o, ref["o"][0][:, i], ref["o"][1][:, i], 2 * Dk + 16, 0, f"o of token {i}")
    near(state, *ref["state"], 16, 0, "state")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("B,L,heads,Dk,Dv,lens", [(1, 9000, (2, 2, 2), 64, 64, None), (2, 5000, (1, 1, 1), 128, 128, [5000, 2777]),
                                                  (3, 3001, (6, 2, 2), 64, 128, [3001, 0, 700]), (1, 20011, (1, 1, 1), 256, 64, None),
                                                  (1, 4097, (1, 1, 1), 32, 256, None)])
def test_linear_attention_long(B, L, heads, Dk, Dv, lens, io):
    """Sequences whose time axis is split."""
    t = TYPES[io]
    a, go, gso = attention_inputs((B, L, heads, Dk, Dv, True, lens, "slow", "dense"), t, L)
    on = on_gpu(a)
    clean = {k: (None if x is None else x.to(DEV)) for k, x in a.items()}
    ref = R.linear_attention(**clean, go=dev(go), gstate_out=dev(gso))
    o, last = H.linear_attention(**on, return_state=True)
    c, r = count(L, Dk, Dv), 1 if io == "bf16" else 0
    near(o, *ref["o"], c, r, "o")
    near(last, *ref["state"], c, 0, "state")
    got = H.linear_attention_backward(**on, go=spoil(go.to(DEV), a["lengths"]), gstate_out=dev(gso))
    for name in ("gq", "gk", "gv", "gstate"):
        near(got[name], *ref[name], c + 8, 0 if name == "gstate" else r, name)


def test_linear_attention_gradients_by_differences():
    """(f(x + e d) - f(x - e d)) / 2e against the gradients' products with d, in fp32 on a smooth case."""
    r = gen(3)
    B, L, N, Dk, Dv = 1, 70, 2, 16, 24
    a = dict(q=r(B, L, N, Dk), k=r(B, L, N, Dk), v=r(B, L, N, Dv), state=r(B, N, Dk, Dv))
    g, go, gso = -torch.tensor([0.02, 0.5]), r(B, L, N, Dv), r(B, N, Dk, Dv)

    def loss(**k):
        o, s = H.linear_attention(**{n: dev(x) for n, x in k.items() if n != "state"}, log_decay=dev(g), state=dev(k["state"]),
                                  return_state=True)
        return float((o.cpu().double() * go).sum() + (s.cpu().double() * gso).sum())

    got = H.linear_attention_backward(dev(a["q"]), dev(a["k"]), dev(a["v"]), dev(go), dev(g), state=dev(a["state"]), gstate_out=dev(gso))
    size = R.linear_attention(**a, log_decay=g)
    # each loss is a sum of o's and the state's terms, off by c 2^-24 of their sizes at most; the loss is linear in each argument,
    # so the quotient has no other error
    c = count(L, Dk, Dv)
    room = 2 * c * EPS32 * float((size["o"][1] * go.abs()).sum() + (size["state"][1] * gso.abs()).sum())
    for n, gn in (("q", "gq"), ("k", "gk"), ("v", "gv"), ("state", "gstate")):
        d = r(*a[n].shape)
        up, down = dict(a), dict(a)
        up[n], down[n] = a[n] + d, a[n] - d
        quotient = (loss(**up) - loss(**down)) / 2
        # x +- d are up to (1 + |d| / |x|) times as large: 8 covers randn's largest values here
        assert abs(quotient - float((got[gn].cpu().double() * d).sum())) <= 8 * room, n


# ---------------------------------------------------------- rotary positions

@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,L,N,D,R_,far,inverse", [(1, 1, 1, 2, 2, False, False), (2, 3, 5, 64, 64, True, False), (3, 7, 2, 80, 40, False, True),
                                                    (1, 300, 3, 128, 96, True, True), (2, 65, 1, 50, 34, True, False),
                                                    (1, 33, 40, 256, 256, False, False), (2, 2, 3, 7, 6, True, False), (1, 5, 2, 18, 2, True, True)])
def test_rotary(B, L, N, D, R_, far, inverse, interleaved, io):
    t, r = TYPES[io], gen(D + L)
    x = r(B, L, N, D).to(t)
    freq, scale = H.rotary_frequencies(R_, scaling="yarn", factor=4.0, device="cpu")
    pos = torch.arange(L)[None] + (torch.tensor([[2 ** 31 - 400], [-2 ** 31], [1 << 20]])[:B] if far else torch.zeros(B, 1, dtype=torch.long))
    ref = R.rotary(x.double(), freq, pos, scale, interleaved, inverse)
    pos32 = dev(pos.to(torch.int32)) if far else None
    got = H.rotary(dev(x), dev(freq), pos32, scale=scale, interleaved=interleaved, inverse=inverse)
    # turns in fp64: 2^-53 (3 roundings) of up to 2^31 / 2 pi of them, and 2^-25 of half a turn to fp32, times 2 pi; then the sine,
    # the scale and two products
    size = scale * (x.double().abs().amax() * 2)
    near(got, ref, size, 16, 0, "rotary")
    assert torch.equal(got[..., R_:].cpu(), x[..., R_:]), "values that are not turned"
    y = dev(x)
    assert H.rotary(y, dev(freq), pos32, scale=scale, interleaved=interleaved, inverse=inverse, out=y) is y
    assert torch.equal(y, got), "in place"
    if not far and B == 1:
        again = H.rotary(dev(x), dev(freq), torch.arange(L, device=DEV, dtype=torch.int32), scale=scale, interleaved=interleaved, inverse=inverse)
        assert torch.equal(again, got), "shared positions"


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_rotary_strides(io):
    """The query and key heads of a projection's rows, out of place and in place, which leaves the rest of the rows alone; heads first; tokens."""
    t, r = TYPES[io], gen(5)
    B, L, N, D = 2, 37, 3, 48
    rows = dev(r(B, L, 2 * N * D + 31).to(t))
    freq, _ = H.rotary_frequencies(32, device=DEV)
    pos = torch.randint(0, 1 << 20, (B, L), generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    part = rows[..., 5:5 + N * D].unflatten(-1, (N, D))
    want = H.rotary(part.contiguous(), freq, pos)
    assert torch.equal(H.rotary(part, freq, pos), want)
    keep = rows.clone()
    H.rotary(part, freq, pos, out=part)
    assert torch.equal(part, want)
    assert torch.equal(rows[..., :5], keep[..., :5]) and torch.equal(rows[..., 5 + N * D:], keep[..., 5 + N * D:])
    first = keep[..., 5:5 + N * D].unflatten(-1, (N, D)).transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(H.rotary(first, freq, pos), want)
    for i in (0, L - 1):
        assert torch.equal(H.rotary(keep[:, i, 5:5 + N * D].unflatten(-1, (N, D)), freq, pos[:, i].contiguous()), want[:, i])


def test_rotary_turns_back():
    """inverse is the transposed turn: its product with another vector is the gradient's."""
    r = gen(9)
    x, gy = r(2, 11, 3, 64), r(2, 11, 3, 64)
    freq, scale = H.rotary_frequencies(64, scaling="ntk", factor=2.0, device=DEV)
    y = H.rotary(dev(x), freq, scale=1.5)
    gx = H.rotary(dev(gy), freq, scale=1.5, inverse=True)
    # two sums of 64 * 66 products, each within 16 roundings of 2 * 1.5 times the largest values
    room = 2 * 16 * EPS32 * 3 * float((x.abs().max() * gy.abs().sum()))
    assert abs(float((y.cpu().double() * gy).sum() - (gx.cpu().double() * x).sum())) <= room


# ---------------------------------------------------------------- group norm

GROUP = [
    # rows, G, Dg
    (1, 1, 1), (3, 2, 1), (5, 7, 3), (4, 1, 8), (9, 3, 16), (2, 12, 33), (70, 5, 64), (33, 12, 128), (3, 300, 20), (6, 2, 257), (5, 3, 500),
    (4, 2, 513), (3, 1, 1024), (2, 2, 1100), (3, 1, 2048), (2, 1, 4000), (2, 3, 5000), (1, 1, 8192), (3, 2, 8200), (2, 1, 20000), (4100, 1, 32),
]


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ["none", "silu", "gate"])
@pytest.mark.parametrize("rows,G,Dg", GROUP)
def test_group_norm(rows, G, Dg, act, io):
    t, r = TYPES[io], gen(rows + Dg)
    D, eps = G * Dg, 1e-3
    x = (r(rows, D) + 3).to(t)
    affine = (rows + G) % 2 == 0 or act == "silu"
    w, b = (1 + 0.2 * r(D), 0.3 * r(D)) if affine else (None, None)
    z = r(rows, D).to(t) if act == "gate" else None
    gy = r(rows, D).to(t)
    v = leaves(x=x, w=w, b=b, z=z)
    y = R.group_norm(v["x"], G, v["w"], v["b"], v["z"], act == "silu", eps)
    (y * S.up(gy)).sum().backward()
    on = dict(weight=dev(w), bias=dev(b), z=dev(z), silu=act == "silu", eps=eps)
    got = H.group_norm(dev(x), G, **on)
    # sums over a group, at most Dg / 256 words of 8 to a thread and 16 steps across threads: k roundings of the mean (of values of
    # size top, which x - mean takes over), of var, and some 12 for the root, the affine map and the sigmoid
    k = Dg / 256 + 8 + 16
    d = (S.up(x).view(rows, G, Dg) - S.up(x).view(rows, G, Dg).mean(-1, keepdim=True))
    rstd = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    spread = lambda q: q.expand(rows, G, Dg).reshape(rows, D)  # noqa: E731
    top = S.up(x).abs().view(rows, G, Dg).amax(-1, keepdim=True)
    n = (d * rstd).reshape(rows, D)
    # n: k roundings of top times rstd from the mean, and k of itself from var
    nsize = spread(top * rstd) + n.abs()
    wt = S.up(w) if affine else torch.ones(D, dtype=torch.float64)
    bs = S.up(b) if affine else torch.zeros(D, dtype=torch.float64)
    msize = nsize * wt.abs() + bs.abs()
    zs = S.up(z).abs() if act == "gate" else None
    # silu is 1.1 steep at most, and not larger than its argument
    ysize = 1.1 * msize if act == "silu" else msize * zs if act == "gate" else msize
    near(got, y.detach(), ysize, 2 * k + 12, 0, "y")
    g = H.group_norm_backward(dev(x), G, dev(gy), **on)
    gm = S.up(gy).abs() * (1.1 if act == "silu" else 1.0)
    if act == "silu":
        gm = gm + S.up(gy).abs() * 0.5 * msize             # its slope is 0.5 steep at most
    if act == "gate":
        gm = gm * zs
        near(g["gz"], v["z"].grad, S.up(gy).abs() * msize * 1.3, 2 * k + 16, 0, "gz")
    gn = (gm * wt.abs()).view(rows, G, Dg)
    n3 = nsize.view(rows, G, Dg)
    gxsize = rstd * (gn + gn.mean(-1, keepdim=True) + n3 * (gn * n3).mean(-1, keepdim=True))
    near(g["gx"], v["x"].grad, gxsize.reshape(rows, D), 6 * k + 24, 0, "gx")
    if affine:
        sums = rows / 256 + 32 + 16                        # over a workgroup's rows, and over the partials
        near(g["gweight"], v["w"].grad, (gm * nsize).sum(0), 2 * k + 20 + sums, 0, "gweight")
        near(g["gbias"], v["b"].grad, gm.sum(0), 2 * k + 20 + sums, 0, "gbias")
    assert (g["gweight"] is None) == (w is None) and (g["gz"] is None) == (z is None)


# ------------------------------------------------------------- all together

@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_block_of_them(io):
    """A prompt and then tokens, as the block runs them, against a prompt of all tokens."""
    t, r = TYPES[io], gen(17)
    B, L, more, N, D, E = 2, 83, 3, 4, 32, 96
    width = 2 * N * D + N * D + N * D
    x = dev(r(B, L + more, E).to(t))
    Wp, w, b = dev((r(E, width) / E ** 0.5).to(t)), dev(1 + 0.1 * r(N * D)), dev(0.1 * r(N * D))
    freq, f = H.rotary_frequencies(D, scaling="yarn", factor=2.0, device=DEV)
    g = -torch.exp(-1 - torch.arange(N, device=DEV, dtype=torch.float32))

    def split(rows):
        qk, v, z = rows.split((2 * N * D, N * D, N * D), -1)
        return qk.unflatten(-1, (2 * N, D)), v.unflatten(-1, (N, D)), z.contiguous()

    def prompt(n, lengths=None):
        qk, v, z = split(x[:, :n] @ Wp)
        qk = H.rotary(qk, freq, scale=f)
        o, s = H.linear_attention(qk[:, :, :N], qk[:, :, N:], v, g, lengths=lengths, return_state=True)
        return H.group_norm(o.flatten(2), N, w, b, z=z), s

    full, last = prompt(L + more)
    y, s = prompt(L)
    ys = [y]
    for i in range(L, L + more):
        qk, v, z = split(x[:, i] @ Wp)
        qk = H.rotary(qk, freq, torch.full((B,), i, device=DEV, dtype=torch.int32), scale=f)
        o = H.linear_attention_step(qk[:, :N], qk[:, N:], v, s, g)
        ys.append(H.group_norm(o.flatten(1), N, w, b, z=z)[:, None])
    got = torch.cat(ys, 1)
    # both sides are the same formulas: they differ by roundings of the projections (two products of one matrix) and of the outputs
    # on the way, some 8 half steps of values that the norm brings to size 1 (8 at most here) times the gate
    room = 8 * HALF[t] * 8 * 8
    assert float((got.double() - full.double()).abs().max()) <= max(room, 1e-4)
    assert float((s - last).abs().max()) <= max(8 * HALF[t], 1e-5) * float(last.abs().max()) * 4
    _, cut = prompt(L + more, torch.tensor([L, L], device=DEV, dtype=torch.int32))
    _, s0 = prompt(L)
    assert float((cut - s0).abs().max()) <= max(8 * HALF[t], 1e-5) * float(s0.abs().max()) * 4
