"""The state-space block's operators where a value is not finite, a sequence
is empty or a limit is near: what such a value may reach, and what stays the
bits of a call without it."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests import ssm_reference as R
from tests.test_ssm import DEV, EPS32, HALF, TYPES, close, dev, gen, leaves, scan_inputs, scan_on_gpu

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def same(a, b, what):
    """Equal bits, or both None."""
    assert (a is None) == (b is None), what
    if a is not None:
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), what


# -------------------------------------------------------------- residual norm

@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 4097, 4099])
@pytest.mark.parametrize("D", [8, 500, 513, 1024, 1100])
def test_norm_backward_without_eps(rows, D, io):
    """eps = 0 on rows that are not zero: a workgroup's places behind the last row add nothing."""
    if rows > 100 and D > 600:
        rows -= 4096 - 1024
    t, r = TYPES[io], gen(rows + D)
    s, w, gy = r(rows, D).to(t), 1 + 0.2 * r(D), r(rows, D).to(t)
    v = leaves(s=s, w=w)
    (R.rms_norm(v["s"], v["w"], 0.0) * R.up(gy)).sum().backward()
    gx, gw = H.rms_norm_backward(dev(s), dev(w), dev(gy), eps=0.0)
    # the counts of test_rms_norm
    c = (D / 256 + 16) / 2 + 8
    rr = 1 / torch.sqrt((R.up(s) ** 2).mean(-1, keepdim=True))
    big = rr * (R.up(w).abs() * R.up(gy).abs()).amax(-1, keepdim=True) * 4
    close(gx, v["s"].grad, 4 * c + 16, big, "gx")
    close(gw, v["w"].grad, c + 8 + rows / 256 + 16, (R.up(gy).abs() * (R.up(s) * rr).abs()).sum(0), "gw")


# --------------------------------------------------------- short convolution

@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 7, 8, 9, 13, 16])
def test_short_conv_bad_value_reaches_its_own_taps(T, silu, bad):
    """x[t] is read by y[t .. t+T-1] alone, and gy[t] by gx[t-T+1 .. t]."""
    r = gen(T)
    B, D, L, at = 2, 5, 70, 37
    x, w, bias, gy = r(B, D, L), r(D, T), r(D), r(B, D, L)
    clean = H.short_conv(dev(x), dev(w), dev(bias), silu=silu)
    gclean = H.short_conv_backward(dev(x), dev(w), dev(gy), dev(bias), silu=silu)
    xb, gb = x.clone(), gy.clone()
    xb[1, 2, at], gb[1, 2, at] = bad, bad
    got = H.short_conv(dev(xb), dev(w), dev(bias), silu=silu)
    reach = torch.zeros(B, D, L, dtype=torch.bool)
    reach[1, 2, at:at + T] = True
    same(got.cpu()[~reach], clean.cpu()[~reach], "y elsewhere")
    if bad != bad:
        assert bool(got.cpu()[reach].isnan().all())
    else:
        assert not bool((got.cpu()[reach].abs() < 1e30).any() and not silu)
    # the loss's gradient: through gy, taps ahead of it
    g = H.short_conv_backward(dev(x), dev(w), dev(gb), dev(bias), silu=silu)
    reach = torch.zeros(B, D, L, dtype=torch.bool)
    reach[1, 2, max(0, at - T + 1):at + 1] = True
    same(g[0].cpu()[~reach], gclean[0].cpu()[~reach], "gx elsewhere, a bad gy")
    assert not bool(g[0].cpu()[reach].isfinite().any())
    keep = [d for d in range(D) if d != 2]
    same(g[1][keep], gclean[1][keep], "gw of other channels")
    # through x: nothing of gx without an activation, and the taps on both sides of it with one
    g = H.short_conv_backward(dev(xb), dev(w), dev(gy), dev(bias), silu=silu)
    reach = torch.zeros(B, D, L, dtype=torch.bool)
    if silu:
        reach[1, 2, max(0, at - T + 1):at + T] = True
    same(g[0].cpu()[~reach], gclean[0].cpu()[~reach], "gx elsewhere, a bad x")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("T", [2, 4, 7, 16])
def test_short_conv_empty_sequence_with_any_state(T, silu, io):
    """A sequence of no steps hands its state on and adds nothing to a gradient, whatever the state holds."""
    t, r = TYPES[io], gen(T)
    B, D, L = 3, 6, 40
    x, w, bias, gy = r(B, D, L).to(t), r(D, T), r(D), r(B, D, L).to(t)
    state, gso = r(B, D, T - 1).to(t), r(B, D, T - 1).to(t)
    lengths = dev(torch.tensor([0, 40, 3], dtype=torch.int32))
    bad = state.clone()
    bad[0, ::2], bad[0, 1::2] = NAN, INF
    out = []
    for s in (state, bad):
        y, last = H.short_conv(dev(x), dev(w), dev(bias), silu=silu, state=dev(s), lengths=lengths, return_state=True)
        same(last[0], dev(s)[0], "the state of an empty sequence")
        out.append((y, *H.short_conv_backward(dev(x), dev(w), dev(gy), dev(bias), silu=silu, state=dev(s), lengths=lengths,
                                              gstate_out=dev(gso))))
    for name, a, b in zip(("y", "gx", "gw", "gbias", "gstate"), *out):
        same(a, b, name)
    same(out[0][4][0], dev(gso)[0], "gstate of an empty sequence")


# ------------------------------------------------------------ selective scan

GRADS = ("gu", "gdelta", "gA", "gB", "gC", "gskip", "gz", "gdelta_bias", "gstate")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("D,G,N,L", [(6, 2, 5, 60), (18, 1, 40, 60), (6, 2, 16, 300), (40, 1, 40, 300), (4, 1, 16, 2100)])
def test_selective_scan_empty_sequence_with_any_state(D, G, N, L, io):
    """A sequence of no steps hands its state on and adds nothing to a gradient, whatever the state holds."""
    t, r = TYPES[io], gen(N + L)
    B = 3
    a, lengths, _ = scan_inputs((B, D, G, N, L, True, True, True, True, True, [L, 0, L // 2]), t, L)
    gy, gso = dev(r(B, D, L).to(t)), dev(r(B, D, N))
    out = []
    for bad in (False, True):
        if bad:
            a["state"][1, ::2], a["state"][1, 1::2] = NAN, INF
        on = scan_on_gpu(a, lengths, True)
        y, h = H.selective_scan(**on, return_state=True)
        same(h[1], on["state"][1], "the state of an empty sequence")
        out.append((y, H.selective_scan_backward(**on, gy=gy, gstate_out=gso)))
    same(out[0][0], out[1][0], "y")
    for k in GRADS:
        same(out[0][1][k], out[1][1][k], k)
    same(out[0][1]["gstate"][1], gso[1], "gstate of an empty sequence")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("D,G,N,L", [(6, 2, 5, 60), (18, 1, 40, 60), (6, 2, 16, 300), (40, 1, 40, 300)])
def test_selective_scan_gradients_behind_a_length_are_zeros(D, G, N, L, io):
    """Also behind a sequence whose own values, or whose later gradient, are not finite."""
    t, r = TYPES[io], gen(N * L)
    B = 2
    lens = [L - 30, 20]
    a, lengths, _ = scan_inputs((B, D, G, N, L, True, True, True, True, True, lens), t, L)
    gy, gso = dev(r(B, D, L).to(t)), r(B, D, N)
    for where in ("u", "state", "gstate_out"):
        b, g = {k: v.clone() for k, v in a.items()}, gso.clone()
        if where == "gstate_out":
            g[:, 1] = NAN
        elif where == "u":
            b["u"][0, 1, L - 32], b["u"][1, 1, 3] = NAN, INF
        else:
            b["state"][:, 1] = INF
        on = scan_on_gpu(b, lengths, True)
        y = H.selective_scan(**on)
        out = H.selective_scan_backward(**on, gy=gy, gstate_out=dev(g))
        for i, n in enumerate(lens):
            assert not bool((y[i, :, n:] != 0).any()), (where, "y")
            for k in ("gu", "gdelta", "gz", "gB", "gC"):
                assert not bool((out[k][i, ..., n:] != 0).any()), (where, k)


# -------------------------------------------------------------- 8-bit product

def e4m3(x):
    return dev(x.clamp(-448, 448)).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("kind", ["spread", "cancelling", "outliers"])
@pytest.mark.parametrize("M,N,K", [(16, 96, 256), (300, 200, 400), (2100, 1700, 128)])
def test_scaled_matmul_sums_of_unlike_sizes(M, N, K, kind):
    """Products of very different sizes, and sums that cancel.  The 8-bit instructions behind a bf16 output of more
    than 64 rows add up 8 neighbouring products at 2^-13 of the largest of them (each of the other 7 loses less than
    that, cut towards zero), and those sums as fp32 does; other sums are fp32 throughout."""
    r = gen(M + K)
    x, w = r(M, K), r(N, K)
    if kind == "spread":
        x, w = x * torch.exp(2 * r(M, K)), w * torch.exp(2 * r(N, K))
    elif kind == "cancelling":
        x, w = 4 * x, 4 * w
        x[:, 1::2], w[:, 1::2] = -x[:, 0::2], w[:, 0::2] * 1.25
    else:
        x[:, ::37] *= 400
        w[:, ::37] *= 100 * torch.sign(r(1, len(range(0, K, 37))))
    q, wq = e4m3(x), e4m3(w)
    kb = -(-K // 128)
    s, ws = torch.exp(r(M, kb)), torch.exp(r(-(-N // 128), kb))
    left = q.double() * dev(s).double().repeat_interleave(128, 1)[:, :K]
    right = wq.double() * dev(ws).double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref = left @ right.t().contiguous()
    size = left.abs() @ right.abs().t().contiguous()
    lost = torch.zeros_like(ref)
    for k in range(0, K, 8):
        lost += (left[:, None, k:k + 8] * right[None, :, k:k + 8]).abs().amax(2)
    lost *= 7 * 2.0 ** -13
    for t in (torch.float32, torch.bfloat16):
        got = H.scaled_matmul(q, dev(s), wq, dev(ws), out_dtype=t).double()
        # K products and 2 K / 128 + 8 roundings of scaled block sums, as in test_scaled_matmul
        room = HALF[t] * ref.abs() + (K + 2 * K / 128 + 8) * EPS32 * size
        if t == torch.bfloat16 and M > 64:
            room += lost
        off = float(((got - ref).abs() / room).max())
        assert off <= 1, (t, off)


def test_scaled_matmul_of_few_rows_sums_in_fp32():
    """Up to 64 rows a bf16 output is the fp32 sum, rounded once, also where the sums cancel."""
    r = gen(21)
    N, K = 200, 400
    for M in (1, 16, 33, 64):
        x, w = 4 * r(M, K), 4 * r(N, K)
        x[:, 1::2], w[:, 1::2] = -x[:, 0::2], w[:, 0::2] * 1.25
        q, wq = e4m3(x), e4m3(w)
        s, ws = dev(torch.exp(r(M, 4))), dev(torch.exp(r(2, 4)))
        got = H.scaled_matmul(q, s, wq, ws)
        # the same sums in the same order, so the same value before the output's rounding
        same(got, H.scaled_matmul(q, s, wq, ws, out_dtype=torch.float32).to(torch.bfloat16), M)


def test_scaled_matmul_more_rows_than_a_sequence_holds():
    """A left of [M, K] counts its rows together: M beyond the longest sequence's 2^22 steps."""
    M, N, K = (1 << 22) + 77, 32, 16
    g = torch.Generator(device=DEV).manual_seed(5)
    q, s = H.quantize(torch.randn(M, K, generator=g, device=DEV))
    wq, ws = H.quantize(torch.randn(N, K, generator=g, device=DEV), 128)
    got = H.scaled_matmul(q, s, wq, ws)
    assert got.shape == (M, N)
    for lo, hi in ((0, 300), (M - 300, M)):
        # tiles of other sizes hold the same sums of one block
        same(got[lo:hi], H.scaled_matmul(q[lo:hi].contiguous(), s[lo:hi].contiguous(), wq, ws), (lo, hi))
    with pytest.raises(H.HyenaError) as e:
        H.scaled_matmul(q, s, wq, ws, channel_major=True)     # there the rows are one sequence
    assert e.value.code == 2


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("B,L,N,K", [(300, 1, 130, 272), (97, 3, 200, 128), (41, 7, 77, 400), (600, 13, 300, 144),
                                     (9000, 1, 3400, 128), (30, 2, 40, 64), (1, 64, 33, 48), (64, 1, 33, 48)])
def test_scaled_matmul_channel_major_of_short_sequences(B, L, N, K, io):
    """Sequences shorter than a word of outputs: the row-major call's bits, in the other order."""
    r = gen(B + L)
    q, s = H.quantize(dev(r(B, L, K)))
    wq, ws = H.quantize(dev(r(N, K)), 128)
    call = lambda cm: H.scaled_matmul(q, s, wq, ws, bias=bias, out_dtype=TYPES[io], channel_major=cm)  # noqa: E731
    bias = dev(r(N))
    same(call(True), call(False).transpose(1, 2).clone(memory_format=torch.contiguous_format), "channel-major")


@pytest.mark.parametrize("L,at", [(60, 33), (300, 171), (2100, 1500)])
@pytest.mark.parametrize("key", ["u", "delta", "z", "Bm", "Cm", "gy"])
def test_selective_scan_bad_value_reaches_its_own_terms(key, L, at):
    """A NaN at a step changes no bit of another sequence, of a channel that does not read it, of the steps before it
    (forward), or of the steps behind it (gradients that come from later steps only)."""
    B, D, G, N = 2, 20, 2, 16
    a, _, _ = scan_inputs((B, D, G, N, L, True, True, True, True, True, None), torch.float32, 9)
    a["gy"], a["gstate_out"] = gen(4)(B, D, L), gen(5)(B, D, N)

    def run(v):
        on = scan_on_gpu({k: t for k, t in v.items() if not k.startswith("g")}, None, True)
        y, h = H.selective_scan(**on, return_state=True)
        return dict(H.selective_scan_backward(**on, gy=dev(v["gy"]), gstate_out=dev(v["gstate_out"])), y=y, h=h)

    clean = run(a)
    bad = dict(a, **{key: a[key].clone()})
    of_group = key in ("Bm", "Cm")
    bad[key][(1, 1, 3, at) if of_group else (1, 13, at)] = NAN
    got = run(bad)
    mine = list(range(10, 20)) if of_group else [13]
    other = [d for d in range(D) if d not in mine]
    for k in ("y", "h", "gu", "gdelta", "gz", "gstate"):
        same(got[k][0], clean[k][0], k)
        same(got[k][1, other], clean[k][1, other], k)
    for k in ("gB", "gC"):
        same(got[k][0], clean[k][0], k)
        same(got[k][1, 0], clean[k][1, 0], k)
    for k in ("gA", "gskip", "gdelta_bias"):
        same(got[k][other], clean[k][other], k)
    same(got["y"][1, :, :at], clean["y"][1, :, :at], "y before")
    if key in ("z", "Cm"):
        same(got["y"][..., at + 1:], clean["y"][..., at + 1:], "y behind")
        same(got["h"], clean["h"], "the state")
    if key == "u":
        same(got["gu"], clean["gu"], "gu")
        same(got["gstate"], clean["gstate"], "gstate")
    if key in ("z", "gy"):
        for k in ("gu", "gB", "gz"):
            same(got[k][..., at + 1:], clean[k][..., at + 1:], k)
