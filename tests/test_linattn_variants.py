"""Linear attention in every width of its kernels: scales and growing states,
what a value that is not finite reaches, and the block's operators in a row,
each against its definition on the values that it was given."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests import linattn_reference as R
from tests.test_linattn import count, near
from tests.test_linattn_rounding import off_by_its_rounding
from tests.test_ssm import DEV, TYPES, dev, gen
from tests.test_ssm_edges import same

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

# L, heads of q k v, Dk, Dv: one, two and four tiles of columns, with 4 and 8 waves, one and two tiles to a wave; heads that are no
# whole words; a split time axis
WIDTHS = [(131, (2, 2, 2), 64, 64), (131, (2, 1, 1), 64, 128), (131, (2, 2, 2), 128, 128), (100, (1, 1, 2), 128, 64),
          (99, (2, 2, 2), 256, 64), (100, (1, 1, 1), 200, 256), (131, (2, 2, 1), 33, 129), (70, (1, 1, 1), 130, 50),
          (900, (2, 1, 1), 128, 128), (700, (1, 1, 1), 64, 96), (600, (2, 2, 2), 40, 33), (700, (1, 1, 1), 256, 24)]


def inputs(L, heads, Dk, Dv, t, seed, B=1):
    r, N = gen(seed), max(heads)
    q, k, v, go = (dev(r(B, L, h, d).to(t)) for h, d in ((heads[0], Dk), (heads[1], Dk), (heads[2], Dv), (N, Dv)))
    return q, k, v, go, dev(r(B, N, Dk, Dv)), dev(r(B, N, Dk, Dv))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("scale,decay", [(0.37, -0.01), (-3.0, -0.2), (0.0, -0.05), (1.0, 0.02), (0.25, 0.004)])
@pytest.mark.parametrize("L,heads,Dk,Dv", WIDTHS[:4] + WIDTHS[8:10])
def test_scales_and_growing_states(L, heads, Dk, Dv, scale, decay, io):
    t, N = TYPES[io], max(heads)
    q, k, v, go, state, gso = inputs(L, heads, Dk, Dv, t, L + Dk)
    g = torch.full((N,), decay, device=DEV)
    ref = R.linear_attention(q, k, v, g, scale, state, go=go, gstate_out=gso)
    # terms of a growing state do not shrink on their way: their sizes are the same formulas of the sizes of the inputs
    sizes = R.linear_attention(*(x.abs() for x in (q, k, v)), g, abs(scale), state.abs(), go=go.abs(), gstate_out=gso.abs())
    o, last = H.linear_attention(q, k, v, g, scale, state, return_state=True)
    got = H.linear_attention_backward(q, k, v, go, g, scale, state, gstate_out=gso)
    # beside the roundings that count() has, an exponent's: exp(X) of relative error X 2^-24, X = |decay| L in all
    c = count(L, Dk, Dv) + 8 + abs(decay) * L
    size = lambda name: torch.maximum(sizes[name][0], ref[name][1]) if decay > 0 else ref[name][1]  # noqa: E731
    for name, x in (("o", o), ("state", last), *got.items()):
        off_by_its_rounding(x, ref[name][0], size(name), c, name)
    for i in range(3):                                  # tokens
        s = state.clone()
        one = H.linear_attention_step(q[:, i], k[:, i], v[:, i], s, g, scale)
        a = [x[:, i:i + 1] for x in (q, k, v)]
        r1 = R.linear_attention(*a, g, scale, state)
        z1 = R.linear_attention(*(x.abs() for x in a), g, abs(scale), state.abs())
        near(one, r1["o"][0][:, 0], z1["o"][0][:, 0], 2 * Dk + 16, 0, "o of a token")
        near(s, r1["state"][0], z1["state"][0], 16, 0, "state of a token")


def places(L):
    return [t for t in (0, 21, 63, 80, 300, 511, L - 1) if t < L]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("L,heads,Dk,Dv", WIDTHS)
def test_bad_value_in_every_width(L, heads, Dk, Dv, which, io):
    """q[t] is read by o[t] alone, k[t] by o from t on, v[t] by one value of o from t on, in the heads that share it.  All else
    keeps its bits."""
    N = max(heads)
    q, k, v, _, state, _ = inputs(L, heads, Dk, Dv, TYPES[io], L + Dv)
    a = dict(q=q, k=k, v=v)
    g = -torch.tensor([0.01, 0.1], device=DEV)[:N]
    clean, last = H.linear_attention(**a, log_decay=g, state=state, return_state=True)
    h, d = a[which].shape[2] - 1, a[which].shape[3] - 7
    share = N // a[which].shape[2]
    for i, at in enumerate(places(L)):
        b = dict(a, **{which: a[which].clone()})
        b[which][0, at, h, d] = (NAN, INF, -INF)[i % 3]
        o, s = H.linear_attention(**b, log_decay=g, state=state, return_state=True)
        reach, behind = torch.zeros_like(o, dtype=torch.bool), torch.zeros_like(s, dtype=torch.bool)
        mine = slice(h * share, (h + 1) * share)
        reach[0, at:at + 1 if which == "q" else L, mine, d if which == "v" else slice(None)] = True
        if which == "k":
            behind[0, mine, d] = True
        if which == "v":
            behind[0, mine, :, d] = True
        same(o[~reach], clean[~reach], f"o elsewhere, {at}")
        same(s[~behind], last[~behind], f"state elsewhere, {at}")
        assert not bool(o[reach].isfinite().any()) and not bool(s[behind].isfinite().any()), at


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("which", ["q", "k", "v", "go"])
@pytest.mark.parametrize("L,heads,Dk,Dv", [(L, (max(h),) * 3, Dk, Dv) for L, h, Dk, Dv in WIDTHS])
def test_bad_value_in_every_width_backward(L, heads, Dk, Dv, which, io):
    """S holds k and v of earlier tokens, G q and go of later ones: gq[t] = S[t] go[t], gk[t] = G[t] v[t], gv[t] = G[t]^T k[t]."""
    N = heads[0]
    q, k, v, go, state, gso = inputs(L, heads, Dk, Dv, TYPES[io], L + Dv)
    a = dict(q=q, k=k, v=v, go=go)
    g = -torch.tensor([0.01, 0.1], device=DEV)[:N]
    clean = H.linear_attention_backward(**a, log_decay=g, state=state, gstate_out=gso)
    d = a[which].shape[3] - 7
    every = slice(None)
    for i, at in enumerate(places(L)):
        b = dict(a, **{which: a[which].clone()})
        b[which][0, at, N - 1, d] = (NAN, INF, -INF)[i % 3]
        got = H.linear_attention_backward(**b, log_decay=g, state=state, gstate_out=gso)
        own, on, up = slice(at, at + 1), slice(at, None), slice(0, at + 1)
        reach = {"go": {"gq": (own, every), "gk": (up, every), "gv": (up, d), "gstate": (every, d)},
                 "v": {"gk": (own, every), "gq": (on, every)},
                 "k": {"gv": (own, every), "gq": (on, d)},
                 "q": {"gk": (up, d), "gv": (up, every), "gstate": (d, every)}}[which]
        for name, x in got.items():
            where = torch.zeros_like(x, dtype=torch.bool)
            if name == "gstate" and name in reach:
                where[0, N - 1, reach[name][0], reach[name][1]] = True
            elif name in reach:
                where[0, reach[name][0], N - 1, reach[name][1]] = True
            same(x[~where], clean[name][~where], f"{name} elsewhere, {which} of {at}")
            assert not bool(x[where].isfinite().any()), (name, at)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_block_by_its_definitions(io):
    """Rotary in place on a projection's rows, attention, norm with a gate, then tokens: each against its definition on what it was
    given, so that every one is held to its own rounding."""
    t, r = TYPES[io], gen(21)
    B, L, N, D = 2, 150, 4, 64
    n = torch.tensor([150, 90], dtype=torch.int32, device=DEV)
    rows, w, b = dev(r(B, L, 4 * N * D).to(t)), dev(1 + 0.1 * r(N * D)), dev(0.1 * r(N * D))
    freq, f = H.rotary_frequencies(D, scaling="yarn", factor=2.0, device=DEV)
    g = -torch.exp(-2 - torch.arange(N, device=DEV, dtype=torch.float32))
    qk, v, z = rows.split((2 * N * D, N * D, N * D), -1)
    qk, v, z = qk.unflatten(-1, (2 * N, D)), v.unflatten(-1, (N, D)), z.contiguous()
    keep = qk.clone()
    pos = torch.arange(L, device=DEV).expand(B, L)
    H.rotary(qk, freq, scale=f, out=qk)
    # the angle's rounding to 2^-25 of half a turn, times pi; sine, scale and two products, as the rotary tests count them
    off_by_its_rounding(qk, R.rotary(keep.double(), freq, pos, f), 2 * f * keep.double().abs().amax(), 16, "rotary")
    q, k = qk[:, :, :N], qk[:, :, N:]
    o, s = H.linear_attention(q, k, v, g, lengths=n, return_state=True)
    ref = R.linear_attention(q, k, v, g, lengths=n)
    c = count(L, D, D)
    off_by_its_rounding(o, *ref["o"], c, "o")
    off_by_its_rounding(s, *ref["state"], c, "state")

    def normed(o, z, y):
        rows = lambda x: x.reshape(-1, N * D).double()  # noqa: E731
        want = R.group_norm(rows(o), N, w.double(), b.double(), rows(z))
        x = rows(o).view(-1, N, D)
        x = x - x.mean(-1, keepdim=True)
        rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)
        top = rows(o).abs().view(-1, N, D).amax(-1, keepdim=True)
        size = ((top + x.abs()) * rstd).reshape(-1, N * D) * w.abs() + b.abs()
        # k roundings of the mean and of var, D / 256 + 24 of them, and some 12 for the root, the affine map and the gate
        off_by_its_rounding(rows(y).to(y.dtype), want, size * rows(z).abs(), 2 * (D / 256 + 24) + 12, "norm")

    normed(o, z, H.group_norm(o.flatten(2), N, w, b, z=z))
    for i in range(3):                                  # tokens, each on the states that the last left
        row, at = dev(r(B, 3 * N, D).to(t)), n + i
        kept = row.clone()
        turned = row[:, :2 * N]
        H.rotary(turned, freq, at, scale=f, out=turned)
        off_by_its_rounding(turned[:, None], R.rotary(kept[:, None, :2 * N].double(), freq, at[:, None], f),
                            2 * f * kept.double().abs().amax(), 16, "rotary of a token")
        before = s.clone()
        one = H.linear_attention_step(turned[:, :N], turned[:, N:], row[:, 2 * N:], s, g)
        ref = R.linear_attention(turned[:, None, :N], turned[:, None, N:], row[:, None, 2 * N:], g, state=before)
        off_by_its_rounding(one[:, None], *ref["o"], 2 * D + 16, "o of a token")
        off_by_its_rounding(s, *ref["state"], 16, "state of a token")
        gate = dev(r(B, N * D).to(t))
        normed(one, gate, H.group_norm(one.flatten(1), N, w, b, z=gate))
