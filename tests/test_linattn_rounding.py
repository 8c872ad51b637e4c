"""Linear attention in bf16 against the float64 definitions, to the outputs' own
rounding: what the matrix products leave of an fp32 value (a state, the weight
of a pair of tokens) is bounded by the sizes of the terms, not by the output.
Inputs where the terms cancel show what is lost there."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests import linattn_reference as R
from tests.test_linattn import count
from tests.test_ssm import DEV, EPS32, TYPES, dev, gen

pytestmark = pytest.mark.gpu


def off_by_its_rounding(got, ref, size, c, what):
    """Each value is round(x) with |x - ref| <= e, e = (p + c 2^-24) size: c fp32 roundings of a term, and in bf16 p = 2^-17
    for a factor of a term taken as the sum of two bf16 values (2^-8 of it is left after the first, 2^-9 of that after the
    second, whose step the remainder fits).  Nothing is nearer to x than round(x), so |got - x| <= |round(ref) - x|, and
    |got - ref| <= |round(ref) - ref| + 2 e."""
    t = got.dtype
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    e = ((2.0 ** -17 if t is torch.bfloat16 else 0.0) + c * EPS32) * size
    own = (ref.to(t).double() - ref).abs()
    off = ((got.double() - ref).abs() - own) / (2 * e + 1e-37)
    assert float(off.max()) <= 1, f"{what}: {float(off.max()):.3g} times its tolerance beyond its own rounding"


def inputs(B, L, heads, Dk, Dv, kind, t, seed):
    """random: no mean anywhere; keys, queries: a direction that the one share and the other lack, so that the terms of o and gv
    cancel; values: one that v shares and go lacks, for gq and gk; means: all of them off zero, but for go."""
    r = gen(seed)
    Hq, Hk, Hv = heads
    q, k, v, go = r(B, L, Hq, Dk), r(B, L, Hk, Dk), r(B, L, Hv, Dv), r(B, L, max(heads), Dv)

    def along(D):
        d = torch.ones(D)
        d[1::2] = -1
        return d

    def without(x):                                     # what is left of x's part along the direction is its rounding's
        d = along(x.shape[-1])
        return x - (x * d).sum(-1, keepdim=True) / d.numel() * d

    if kind == "keys":
        q, k = without(q), k + 4 * along(Dk)
    elif kind == "queries":
        q, k = q + 4 * along(Dk), without(k)
    elif kind == "values":
        go, v = without(go), v + 4 * along(Dv)
    elif kind == "means":
        q, k, v, go = q + 1, k + 1, v + 1, go - go.mean(-1, keepdim=True)
    state, gso = r(B, max(heads), Dk, Dv), r(B, max(heads), Dk, Dv)
    return [dev(x.to(t)) for x in (q, k, v, go)], dev(state), dev(gso)


SIZES = [
    # B, L, heads of q k v, Dk, Dv, lengths: a block and less, where the block's own tokens make most of an output up; several
    # blocks; a split time axis; every width of a workgroup's columns and of a head, odd ones among them
    (2, 17, (1, 1, 1), 16, 16, None), (1, 64, (2, 2, 2), 64, 64, None), (1, 500, (2, 2, 2), 64, 64, None),
    (1, 700, (1, 1, 1), 64, 128, None), (2, 450, (1, 1, 1), 128, 128, [450, 131]), (1, 260, (2, 1, 1), 128, 64, None),
    (1, 300, (1, 1, 1), 256, 64, None), (1, 280, (1, 1, 1), 200, 256, None), (1, 321, (1, 1, 1), 40, 33, None),
    (1, 1500, (4, 2, 2), 96, 80, [1337]),
]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["random", "keys", "queries", "values", "means"])
@pytest.mark.parametrize("B,L,heads,Dk,Dv,lens", SIZES)
def test_outputs_are_off_by_their_own_rounding(B, L, heads, Dk, Dv, lens, kind, io):
    (q, k, v, go), state, gso = inputs(B, L, heads, Dk, Dv, kind, TYPES[io], L + Dv)
    g = dev(-torch.tensor([1e-3, 1e-4, 0.02, 0.3])[:max(heads)])
    n = None if lens is None else dev(torch.tensor(lens, dtype=torch.int32))
    ref = R.linear_attention(q, k, v, g, state=state, lengths=n, go=go, gstate_out=gso)
    o, last = H.linear_attention(q, k, v, g, state=state, lengths=n, return_state=True)
    got = H.linear_attention_backward(q, k, v, go, g, state=state, lengths=n, gstate_out=gso)
    c = count(L, Dk, Dv)
    off_by_its_rounding(o, *ref["o"], c, "o")
    off_by_its_rounding(last, *ref["state"], c, "state")
    for name in ("gq", "gk", "gv", "gstate"):
        off_by_its_rounding(got[name], *ref[name], c + 8, name)


@pytest.mark.parametrize("kind", ["random", "keys", "values", "means"])
@pytest.mark.parametrize("L,Dk,Dv", [(2048, 64, 128), (4100, 128, 128), (2000, 64, 64), (2000, 256, 64)])
def test_bf16_errors_by_spans(L, Dk, Dv, kind):
    """The norm of the error over spans of 256 tokens of a long sequence, whose outputs come from the state: that of the
    outputs' own rounding, and of what is left of the factors.  A rounding of the state's Dk values loses parts of their
    products with q that are independent of each other: sqrt(Dk) and not Dk times the largest, and 4 for the largest over
    the typical one; the same in fp32 for c roundings."""
    N = 2
    (q, k, v, go), _, _ = inputs(1, L, (N, N, N), Dk, Dv, kind, torch.bfloat16, L)
    g = dev(torch.tensor([-1e-3, -1e-2]))
    ref = R.linear_attention(q, k, v, g, go=go)
    got = H.linear_attention_backward(q, k, v, go, g)
    got["o"] = H.linear_attention(q, k, v, g)
    c = count(L, Dk, Dv) + 8
    for name in ("o", "gq", "gk", "gv"):
        x, (f, z) = got[name].double(), ref[name]
        for h in range(N):
            for s in range(0, L, 256):
                part = (0, slice(s, s + 256), h)
                error, own = (x[part] - f[part]).norm(), (f[part].to(torch.bfloat16).double() - f[part]).norm()
                room = 4 * (2.0 ** -17 + c * EPS32) / min(Dk, Dv) ** 0.5 * z[part].norm()
                assert float(error) <= float((own ** 2 + room ** 2).sqrt()) * 1.01, (name, h, s, float(error / own))
