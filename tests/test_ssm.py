"""The state-space block's operators on the GPU against their float64
definitions (tests/ssm_reference.py), values and gradients, at the sizes and
masks where tiles, words and segments end.

Tolerances.  An output is compared within

    half * |ref| + c * 2^-24 * size,

half the I/O dtype's half step (2^-8 bf16, 2^-24 fp32: one rounding where the
value is stored) and size the sum of the sizes of the terms that make it up,
bounded per tensor by its largest value times a count: fp32 arithmetic puts a
relative error of at most 2^-24 (twice that for the exponential, the
reciprocal and the square root) on each of the c operations that a term
passes through.  c is counted at each test."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests import ssm_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
EPS32 = 2.0 ** -24


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return lambda *n: torch.randn(*n, generator=g)


def dev(t):
    return None if t is None else t.to(DEV)


def close(got, ref, c, size=None, what=""):
    """got within half a step of ref and c fp32 roundings of terms of `size` (default: the largest |ref|)."""
    got64 = got.detach().to("cpu", torch.float64)
    assert got64.shape == ref.shape, (what, got64.shape, ref.shape)
    assert bool(torch.isfinite(got64).all()), f"{what}: not finite"
    if not ref.numel():
        return
    if size is None:
        size = ref.abs().max()
    room = HALF[got.dtype] * ref.abs() + c * EPS32 * size + 1e-37
    off = (got64 - ref).abs() / room
    assert float(off.max()) <= 1, f"{what}: {float(off.max()):.3g} times its tolerance"


def spoil(t, lengths):
    """NaN and infinities behind each sequence's length."""
    if lengths is None:
        return t
    t = t.clone()
    L = t.shape[-1]
    for b, n in enumerate(R.clamp_lengths(lengths, t.shape[0], L)):
        t[b, ..., n:] = float("nan")
        if n < L:
            t[b, ..., L - 1] = float("inf")
    return t


def leaves(**kw):
    """Float64 leaves with gradients for the tensors that are there."""
    out = {k: R.up(v) for k, v in kw.items()}
    for v in out.values():
        if v is not None:
            v.requires_grad_(True)
    return out


# --------------------------------------------------------- short convolution

CONV = [
    # B, D, L, T, silu, bias, state, lengths
    (1, 1, 1, 1, False, False, False, None),
    (2, 3, 1, 4, True, True, True, None),
    (2, 5, 2, 4, True, True, False, [0, 2]),
    (3, 7, 9, 4, True, True, True, [1, 0, 9]),
    (3, 5, 33, 2, False, True, True, [33, 1, 17]),
    (2, 3, 100, 3, True, False, False, [-5, 1000]),
    (2, 4, 257, 5, True, True, True, [256, 3]),
    (2, 3, 130, 8, False, True, True, [130, 5]),
    (4, 2, 61, 16, True, True, True, [61, 15, 16, 2]),
    (1, 2, 2047, 4, True, True, True, None),
    (1, 3, 2049, 4, True, True, False, [2048]),
    (2, 2, 4500, 16, True, True, True, [4500, 2050]),
    (1, 1, 16400, 4, True, True, True, None),           # two partials along a row in the backward
    (33, 17, 24, 4, True, True, False, None),           # many short rows in a workgroup
]


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_short_conv(case, io):
    B, D, L, T, use_silu, has_bias, has_state, lens = case
    t, r = TYPES[io], gen(L * 31 + T)
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    x, w = r(B, D, L).to(t), r(D, T) / T ** 0.5
    bias = r(D) if has_bias else None
    state = r(B, D, T - 1).to(t) if has_state and T > 1 else None
    gy = r(B, D, L).to(t)
    gso = r(B, D, T - 1).to(t) if T > 1 else None
    n = R.clamp_lengths(lengths, B, L)
    v = leaves(x=x, w=w, bias=bias, state=state)
    y, last = R.short_conv(v["x"], v["w"], v["bias"], use_silu, v["state"], lengths)
    loss = (y * R.up(gy)).sum() + ((last * R.up(gso)).sum() if T > 1 else 0)
    loss.backward()

    xs, gys = dev(spoil(x, lengths)), dev(spoil(gy, lengths))
    got, got_last = H.short_conv(xs, dev(w), dev(bias), silu=use_silu, state=dev(state), lengths=dev(lengths),
                                 return_state=True)
    # T products and sums, the bias, and about 8 for the sigmoid, on values up to 1 + sum |w| |x|
    size = 8 + 2 * float((w.abs().sum(1).max() * x.float().abs().max()))
    close(got, y.detach(), T + 10, size, "y")
    assert torch.equal(got_last.cpu(), last.detach().to(t)), "the state left behind is a copy"
    gx, gw, gb, gs = H.short_conv_backward(xs, dev(w), gys, dev(bias), silu=use_silu, state=dev(state),
                                           lengths=dev(lengths), gstate_out=dev(gso))
    # gp: the same again and 6 for the derivative (at most 1.1); then T terms
    g = 1.1 * float(gy.float().abs().max())
    close(gx, v["x"].grad, 3 * T + 24, g * size + (float(gso.float().abs().max()) if T > 1 else 0), "gx")
    # sums over time: a chain of 8 * (span / 2048) terms in a lane, 8 steps of tree, the partials
    terms = 8 * (min(L, 16384) / 2048 + 1) + 16 + B * 2
    total = sum(n) + 1
    close(gw, v["w"].grad, T + 24 + terms, g * size * total ** 0.5 * 4 + g * size, "gw")
    if has_bias:
        close(gb, v["bias"].grad, T + 24 + terms, g * size * total ** 0.5 * 4 + g, "gbias")
    else:
        assert gb is None
    if state is not None:
        close(gs, v["state"].grad, 3 * T + 24, g * size + float(gso.float().abs().max()), "gstate")
    else:
        assert gs is None
    for b in range(B):
        assert not bool(got[b, :, n[b]:].any()) and not bool(gx[b, :, n[b]:].any()), "zeros behind a length"


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 4, 7, 16])
def test_short_conv_in_pieces_and_tokens(T, io):
    """A sequence in one call equals the same in pieces and in single tokens, bit for bit."""
    t, r = TYPES[io], gen(T)
    B, D, L = 3, 21, 40
    x, w, bias = dev(r(B, D, L).to(t)), dev(r(D, T)), dev(r(D))
    whole, last = H.short_conv(x, w, bias, silu=True, return_state=True)
    state = torch.zeros(B, D, T - 1, dtype=t, device=DEV) if T > 1 else None
    parts = []
    for lo, hi in ((0, 1), (1, 9), (9, 30)):
        if T > 1:
            y, state = H.short_conv(x[..., lo:hi].contiguous(), w, bias, silu=True, state=state, return_state=True)
        else:
            y = H.short_conv(x[..., lo:hi].contiguous(), w, bias, silu=True)
        parts.append(y)
    for k in range(30, L):
        parts.append(H.short_conv_step(x[..., k].contiguous(), w, state, bias, silu=True)[..., None])
    assert torch.equal(torch.cat(parts, -1), whole)
    if T > 1:
        assert torch.equal(state, last)


# ------------------------------------------------------------ selective scan

SCAN = [
    # B, D, G, N, L, z, skip, bias, softplus, state, lengths
    (1, 1, 1, 1, 1, False, False, False, True, False, None),
    (2, 3, 1, 16, 1, True, True, True, True, True, None),
    (2, 5, 1, 16, 7, True, True, True, True, True, [0, 7]),
    (2, 16, 2, 4, 8, False, True, True, True, True, [1, 8]),
    (3, 18, 3, 3, 9, True, False, False, True, False, [9, 0, 4]),
    (2, 17, 1, 8, 127, True, True, True, True, True, [127, 100]),
    (1, 33, 1, 11, 128, True, True, True, True, False, None),
    (2, 16, 4, 16, 129, True, True, True, False, True, [129, 128]),
    (2, 10, 2, 17, 300, True, True, True, True, True, [257, 300]),
    (1, 3, 1, 32, 200, True, True, True, True, True, None),
    (1, 5, 1, 33, 150, False, True, True, True, True, [-3]),
    (1, 18, 1, 64, 140, True, True, True, True, True, [139]),
    (2, 4, 1, 16, 1100, True, True, True, True, True, [1100, 600]),    # the time axis split in two
    (1, 2, 1, 5, 2200, True, True, True, True, False, [2100]),
    (1, 2, 1, 3, 5000, True, True, True, True, True, [4700]),          # 40 segments, 40 chunks
    (1, 40, 1, 16, 260, True, True, True, True, True, None),           # several channel tiles
    (2, 4000, 2, 16, 20, True, True, True, True, True, [20, 13]),      # rows enough for a wave to hold all states
]


def scan_inputs(case, t, seed):
    B, D, G, N, L, has_z, has_skip, has_bias, softplus, has_state, lens = case
    r = gen(seed)
    A = -torch.arange(1, N + 1).float() * (0.75 + 0.5 * torch.rand(D, 1, generator=torch.Generator().manual_seed(seed)))
    a = dict(u=r(B, D, L).to(t), delta=(0.5 * r(B, D, L) - (0 if has_bias else 3)).to(t), A=A, Bm=r(B, G, N, L).to(t),
             Cm=r(B, G, N, L).to(t), skip=r(D) if has_skip else None, z=r(B, D, L).to(t) if has_z else None,
             delta_bias=r(D) - 3 if has_bias else None, state=r(B, D, N) if has_state else None)
    if not softplus:                                    # time steps given as they are
        a["delta"] = a["delta"].float().abs().mul(0.1).to(t)
        a["delta_bias"] = a["delta_bias"].abs() * 0.02
    return a, None if lens is None else torch.tensor(lens, dtype=torch.int32), softplus


def scan_on_gpu(a, lengths, softplus):
    on = {k: dev(spoil(v, lengths)) if k in ("u", "delta", "Bm", "Cm", "z") and v is not None else dev(v)
          for k, v in a.items()}
    on.update(softplus=softplus, lengths=dev(lengths))
    return on


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_selective_scan(case, io):
    B, D, G, N, L = case[:5]
    t = TYPES[io]
    a, lengths, softplus = scan_inputs(case, t, L + N)
    n = R.clamp_lengths(lengths, B, L)
    r = gen(L * 7 + N)
    gy, gso = r(B, D, L).to(t), r(B, D, N)
    v = leaves(**a)
    y, h = R.selective_scan(*[v[k] for k in ("u", "delta", "A", "Bm", "Cm", "skip", "z", "delta_bias")], softplus,
                            v["state"], lengths)
    (y * R.up(gy)).sum().add((h * R.up(gso)).sum()).backward()

    on = scan_on_gpu(a, lengths, softplus)
    got, got_h = H.selective_scan(**on, return_state=True)
    # The state's error: each step adds the roundings of its own decay (|dt A| of the exponent's, 3 more) and of its
    # input (about 12 from softplus on), which fade with the state itself: steps that matter are those of a decay, at
    # most min(L, 1 / (1 - a)) ~ 100 for the time steps above.  Sums over N states follow.
    steps = min(L, 100)
    c_h = 16 + 4 * steps
    size_h = float(h.detach().abs().max()) + 1
    m = float(max(v[k].detach().abs().max() for k in ("Cm", "Bm")))
    close(got_h, h.detach(), c_h, size_h, "state")
    size_y = size_h * m * N ** 0.5 * 2 + float(y.detach().abs().max())
    close(got, y.detach(), c_h + N + 16, size_y, "y")
    for b in range(B):
        assert not bool(got[b, :, n[b]:].any()), "zeros behind a length"

    g = H.selective_scan_backward(**on, gy=dev(spoil(gy, lengths)), gstate_out=dev(gso))
    c = 2 * c_h + N + 40                                # both recurrences, the gates and the sums over states
    total = (sum(n) + 1) ** 0.5 * 4                     # sums over batch and time of terms of both signs
    for name, key, extra, many in (("gu", "u", 0, 1), ("gdelta", "delta", 0, 1), ("gz", "z", 0, 1), ("gB", "Bm", D // G, 1),
                                   ("gC", "Cm", D // G, 1), ("gA", "A", L + B, total), ("gskip", "skip", L + B, total),
                                   ("gdelta_bias", "delta_bias", L + B, total), ("gstate", "state", 0, 1)):
        if a[key] is None:
            assert g[name] is None, name
            continue
        ref = v[key].grad if v[key].grad is not None else torch.zeros_like(v[key])    # no step reads it
        # intermediate products are larger than the sums they cancel in by the sizes of the factors
        size = (float(ref.abs().max()) * 4 + 4) * (many if many > 1 else 1)
        close(g[name], ref, c + extra, size, name)
    for b in range(B):
        for k in ("gu", "gdelta", "gz", "gB", "gC"):
            if g[k] is not None:
                assert not bool(g[k][b, ..., n[b]:].any()), f"{k}: zeros behind a length"


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("N,G", [(1, 1), (4, 2), (11, 1), (16, 1), (64, 3)])
def test_selective_scan_in_pieces_and_tokens(N, G, io):
    """A sequence in one call against the same in pieces and in single tokens."""
    t = TYPES[io]
    B, D, L = 2, 6 * G, 150
    a, _, _ = scan_inputs((B, D, G, N, L, True, True, True, True, True, None), t, N)
    on = scan_on_gpu(a, None, True)
    whole, last = H.selective_scan(**on, return_state=True)
    state, parts = on["state"], []
    cut = lambda lo, hi: {k: on[k][..., lo:hi].contiguous() for k in ("u", "delta", "Bm", "Cm", "z")}  # noqa: E731
    rest = dict(A=on["A"], skip=on["skip"], delta_bias=on["delta_bias"])
    for lo, hi in ((0, 1), (1, 130)):
        y, state = H.selective_scan(**cut(lo, hi), **rest, state=state, return_state=True)
        parts.append(y)
    for k in range(130, L):
        one = {name: v[..., 0].contiguous() for name, v in cut(k, k + 1).items()}
        parts.append(H.selective_scan_step(**one, **rest, state=state)[..., None])
    # the same sums in another order: twice the state's own error, as above
    close(state, last.cpu().double(), 2 * (16 + 4 * 100), float(last.abs().max()) + 1, "state")
    y = torch.cat(parts, -1)
    size = (float(last.abs().max()) + 1) * 4 * N ** 0.5 * 2 + float(whole.float().abs().max())
    off = (y.double() - whole.double()).abs().cpu()
    room = 2 * HALF[t] * whole.double().abs().cpu() + 2 * (16 + 400 + N + 16) * EPS32 * size
    assert bool((off <= room).all())


def test_selective_scan_gradients_against_differences():
    """Directional differences of the float64 loss against the fp32 gradients."""
    case = (2, 6, 2, 7, 140, True, True, True, True, True, [140, 77])
    a, lengths, softplus = scan_inputs(case, torch.float32, 5)
    B, D, G, N, L = case[:5]
    r = gen(6)
    gy, gso = r(B, D, L), r(B, D, N)
    on = scan_on_gpu(a, lengths, softplus)
    g = H.selective_scan_backward(**on, gy=dev(spoil(gy, lengths)), gstate_out=dev(gso))

    def loss(v):
        y, h = R.selective_scan(*[v[k] for k in ("u", "delta", "A", "Bm", "Cm", "skip", "z", "delta_bias")], softplus,
                                v["state"], lengths)
        return float((y * R.up(gy)).sum() + (h * R.up(gso)).sum())

    base, step = {k: R.up(v) for k, v in a.items()}, 1e-5
    for name, key in (("gu", "u"), ("gdelta", "delta"), ("gA", "A"), ("gB", "Bm"), ("gC", "Cm"), ("gskip", "skip"),
                      ("gz", "z"), ("gdelta_bias", "delta_bias"), ("gstate", "state")):
        way = r(*base[key].shape).double()
        ahead, behind = dict(base), dict(base)
        ahead[key], behind[key] = base[key] + step * way, base[key] - step * way
        slope = (loss(ahead) - loss(behind)) / (2 * step)
        along = float((g[name].cpu().double() * way).sum())
        # the difference is off by step^2 times a third derivative and 1e-16 / step; the gradient by some hundred
        # roundings on each of its values, which add up along the direction as a root of sums of squares
        room = 1e-4 * abs(slope) + 600 * EPS32 * float((g[name].cpu().double() * way).norm()) * 8 + 1e-4
        assert abs(along - slope) <= room, (name, along, slope)


def test_selective_scan_one_bad_value_stays_behind_its_step():
    """A NaN input changes nothing before its step, in no other channel and no other sequence."""
    case = (2, 20, 1, 16, 300, True, True, True, True, True, None)
    a, _, _ = scan_inputs(case, torch.float32, 9)
    clean = H.selective_scan(**scan_on_gpu(a, None, True))
    a["u"][1, 3, 171] = float("nan")
    got = H.selective_scan(**scan_on_gpu(a, None, True))
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1, 3, :171], clean[1, 3, :171])
    assert bool(got[1, 3, 171:].isnan().all())
    keep = [d for d in range(20) if d != 3]
    assert torch.equal(got[1, keep], clean[1, keep])


# -------------------------------------------------------------- residual norm

@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 5), (17, 8), (2, 127), (5, 128), (3, 129), (4, 512), (7, 513),
                                    (1030, 40), (5000, 24), (3, 1024), (5, 1025), (2, 2048), (3, 2049), (2, 4097), (3, 8192),
                                    (2, 8200), (5, 20001)])
def test_rms_norm(rows, D, residual, io):
    t, r = TYPES[io], gen(rows + D)
    x, w, gy = r(rows, D).to(t), 1 + 0.2 * r(D), r(rows, D).to(t)
    res = (2 * r(rows, D)).to(t) if residual else None
    gs = r(rows, D).to(t) if residual else None
    if rows > 2:
        x[1] = 0
        if residual:
            res[1] = 0                                  # a row of zeros stays zero
    s = (x.double() + res.double()).to(t) if residual else x
    eps = 1e-5
    v = leaves(s=s, w=w)
    y = R.rms_norm(v["s"], v["w"], eps)
    ((y * R.up(gy)).sum() + ((v["s"] * R.up(gs)).sum() if residual else 0)).backward()
    got = H.rms_norm(dev(x), dev(w), residual=dev(res), eps=eps)
    if residual:
        got, got_s = got
        assert torch.equal(got_s.cpu(), s)
    # a sum of D squares in chains of at most D / 256 + 8 terms and 8 steps of tree, halved by the root; 8 more
    c = (D / 256 + 16) / 2 + 8
    close(got, y.detach(), c, y.detach().abs(), "y")
    gx, gw = H.rms_norm_backward(dev(s), dev(w), dev(gy), gs=dev(gs), eps=eps)
    # gx is a difference of two terms of the size of r |w gy|
    rr = 1 / torch.sqrt((R.up(s) ** 2).mean(-1, keepdim=True) + eps)
    big = rr * (R.up(w).abs() * R.up(gy).abs()).amax(-1, keepdim=True) * 4 + (R.up(gs).abs() if residual else 0)
    close(gx, v["s"].grad, 4 * c + 16, big, "gx")
    close(gw, v["w"].grad, c + 8 + rows / 256 + 16, (R.up(gy).abs() * (R.up(s) * rr).abs()).sum(0), "gw")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 16), (17, 127), (5, 128), (3, 130), (6, 1024), (3, 2050), (2, 8200)])
def test_rms_norm_quantized(rows, D, io):
    t, r = TYPES[io], gen(rows * D)
    x, w, res = r(rows, D).to(t), 1 + 0.2 * r(D), r(rows, D).to(t)
    if rows > 2:
        x[1], res[1] = 0, 0
    s = (x.double() + res.double()).to(t)
    y = R.rms_norm(R.up(s), R.up(w), 1e-6)
    q, scales, got_s = H.rms_norm_quantized(dev(x), dev(w), residual=dev(res), eps=1e-6)
    assert torch.equal(got_s.cpu(), s)
    assert q.dtype == torch.float8_e4m3fn and scales.shape == (rows, -(-D // 128))
    _, ref = R.quantize(y, 1)
    c = (D / 256 + 16) / 2 + 8
    close(scales, ref, c + 2, ref, "scales")
    each = scales.cpu().double().repeat_interleave(128, 1)[:, :D]
    held = q.cpu().double() * each
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 of the scale below 2^-6 of it; and y's own roundings
    room = y.abs() * (2.0 ** -4 + 2 * c * EPS32) + each * 2.0 ** -10 + 1e-37
    assert bool(((held - y).abs() <= room).all())
    q2, scales2 = H.rms_norm_quantized(dev(s), dev(w), eps=1e-6)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(scales2, scales)


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 127), (17, 128), (130, 129), (257, 400), (128, 1024)])
def test_quantize(rows, K, block_rows, io):
    """Codes and scales are what the definition gives, exactly."""
    x = (gen(rows + K)(rows, K) * torch.exp(gen(K)(rows, 1))).to(TYPES[io])
    x[0] = 0
    q, scales = H.quantize(dev(x), block_rows)
    codes, ref = R.quantize(R.up(x), block_rows)
    assert torch.equal(scales.cpu().double(), ref)
    assert torch.equal(q.cpu().double(), codes)


def test_quantize_bad_values_stay_in_their_block():
    x = gen(3)(4, 300)
    clean, cs = H.quantize(dev(x))
    x[1, 130], x[2, 5] = float("nan"), float("inf")
    q, s = H.quantize(dev(x))
    held = q.cpu().float() * s.cpu().repeat_interleave(128, 1)[:, :300]
    assert bool(held[1, 128:256].isnan().all()) and bool(held[2, :128].isnan().all())
    ok = torch.ones(4, 3, dtype=torch.bool)
    ok[1, 1] = ok[2, 0] = False
    assert torch.equal(s.cpu()[ok], cs.cpu()[ok])
    m = ok.repeat_interleave(128, 1)[:, :300]
    assert torch.equal(q.cpu().view(torch.uint8)[m], clean.cpu().view(torch.uint8)[m])


def test_quantize_tiny_values():
    """A block whose scale would be below the least normal number is held at that scale."""
    x = torch.full((1, 128), 2.0 ** -140)
    q, s = H.quantize(dev(x))
    assert float(s) == 2.0 ** -126 and not bool(q.cpu().float().isnan().any())


# -------------------------------------------------------------- 8-bit product

PRODUCT = [(1, 1, 16), (1, 16, 128), (3, 130, 144), (16, 64, 256), (17, 257, 400), (33, 128, 1024), (64, 100, 128),
           (65, 65, 2048), (130, 384, 272), (200, 513, 640), (300, 129, 1040), (520, 260, 256),
           (1800, 1700, 272), (3850, 3333, 144)]              # 128 x 128 and 256 x 256 tiles


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("channel_major", [False, True])
@pytest.mark.parametrize("M,N,K", PRODUCT)
def test_scaled_matmul(M, N, K, channel_major, io):
    r = gen(M + N + K)
    x, w = r(M, K) * torch.exp(r(M, 1)), r(N, K)
    bias = r(N) if M % 2 else None
    q, s = H.quantize(dev(x))
    wq, ws = H.quantize(dev(w), 128)
    ref, size = R.scaled_matmul(q.cpu().double(), R.up(s), wq.cpu().double(), R.up(ws), R.up(bias))
    got = H.scaled_matmul(q, s, wq, ws, bias=dev(bias), out_dtype=TYPES[io], channel_major=channel_major)
    if channel_major:
        got = got.t()
    # fp32 sums of K products and K / 128 scaled ones; the 8-bit instructions behind a bf16 output keep 2^-16
    c = K + 2 * K / 128 + 8 if io == "fp32" else 2.0 ** 8 + 2 * K / 128 + 8
    close(got, ref, c, size, "out")


def test_scaled_matmul_layouts_and_batches():
    r = gen(8)
    B, L, K, N = 3, 37, 160, 200
    q, s = H.quantize(dev(r(B, L, K)))
    wq, ws = H.quantize(dev(r(N, K)), 128)
    rows = H.scaled_matmul(q, s, wq, ws)
    assert rows.shape == (B, L, N) and rows.dtype == torch.bfloat16
    cols = H.scaled_matmul(q, s, wq, ws, channel_major=True)
    assert cols.shape == (B, N, L)
    # the same products and the same order of sums, on the other side of the matrix instruction
    off = (cols.transpose(1, 2).double() - rows.double()).abs()
    assert bool((off <= 2 * HALF[torch.bfloat16] * rows.double().abs() + 2.0 ** -14 * rows.double().abs().max()).all())
    one = H.scaled_matmul(q[1].contiguous(), s[1].contiguous(), wq, ws)
    # few rows are summed in parts along k: each side is within half a step, and 2^-16 of its terms, of the product
    off = (one.double() - rows[1].double()).abs()
    assert bool((off <= 2 * HALF[torch.bfloat16] * rows[1].double().abs() + 2.0 ** -14 * rows.double().abs().max()).all())


# ------------------------------------------------- streams, graphs, together

def block_params(D, E, N, T, t, seed=1):
    """A state-space block of width D, inner width E."""
    r = gen(seed)
    p = dict(norm=1 + 0.1 * r(D), w_in=r(2 * E, D) / D ** 0.5, conv=r(E, T) / T ** 0.5, conv_bias=0.1 * r(E),
             w_bc=(r(2 * N, E) / E ** 0.5).to(t), w_dt=(r(E, E) / E ** 0.5 * 0.1).to(t), dt_bias=r(E) * 0.1 - 3,
             A=-torch.arange(1, N + 1).float().repeat(E, 1), skip=r(E))
    p = {k: dev(v) for k, v in p.items()}
    p["wq"], p["wscales"] = H.quantize(p["w_in"], 128)
    p.update(E=E, N=N, T=T)
    return p


def block_prompt(p, x, residual, lengths, cs=None, ss=None):
    """x [B, L, D] -> (y [B, E, L], the residual stream, the two states)."""
    B, L, D = x.shape
    E, N = p["E"], p["N"]
    q, sc, s = H.rms_norm_quantized(x, p["norm"], residual=residual)
    xz = H.scaled_matmul(q, sc, p["wq"], p["wscales"], out_dtype=x.dtype, channel_major=True)
    u, cs = H.short_conv(xz[:, :E].contiguous(), p["conv"], p["conv_bias"], silu=True, state=cs, lengths=lengths,
                         return_state=True)
    bc = torch.matmul(p["w_bc"], u).view(B, 2, N, L)
    delta = torch.matmul(p["w_dt"], u)
    y, ss = H.selective_scan(u, delta, p["A"], bc[:, :1].contiguous(), bc[:, 1:].contiguous(), skip=p["skip"],
                             z=xz[:, E:].contiguous(), delta_bias=p["dt_bias"], state=ss, lengths=lengths,
                             return_state=True)
    return y, s, cs, ss


def block_token(p, x, residual, cs, ss):
    """One token for each sequence: x [B, D] -> y [B, E]; the states move on."""
    E, N = p["E"], p["N"]
    q, sc, s = H.rms_norm_quantized(x, p["norm"], residual=residual)
    xz = H.scaled_matmul(q, sc, p["wq"], p["wscales"], out_dtype=x.dtype)
    u = H.short_conv_step(xz[:, :E].contiguous(), p["conv"], cs, p["conv_bias"], silu=True)
    bc = torch.matmul(u, p["w_bc"].t()).view(-1, 2, N)
    delta = torch.matmul(u, p["w_dt"].t())
    return H.selective_scan_step(u, delta, p["A"], bc[:, :1].contiguous(), bc[:, 1:].contiguous(), ss, skip=p["skip"],
                                 z=xz[:, E:].contiguous(), delta_bias=p["dt_bias"])


def test_block_prompt_then_tokens():
    """The operators as a serving loop runs them: right-padded prompts in one
    call, then a token at a time, against the whole sequences in one call."""
    t, B, D, E, N, T, L = torch.float32, 3, 64, 96, 8, 4, 50
    p, r = block_params(D, E, N, T, t), gen(2)
    x, res = dev(r(B, L, D)), dev(r(B, L, D))
    whole = block_prompt(p, x, res, None)[0]
    lengths = torch.tensor([40, 1, 33], dtype=torch.int32)
    y, _, cs, ss = block_prompt(p, x, res, dev(lengths))
    for b, n in enumerate(lengths.tolist()):
        # the same operations on the same values; the matrix products may sum in another order
        assert torch.allclose(y[b, :, :n], whole[b, :, :n], rtol=1e-4, atol=1e-4 * float(whole.abs().max()))
    for k in range(10):
        at = lengths.long() + k
        xt = torch.stack([x[b, at[b]] for b in range(B)]).contiguous()
        rt = torch.stack([res[b, at[b]] for b in range(B)]).contiguous()
        got = block_token(p, xt, rt, cs, ss)
        want = torch.stack([whole[b, :, at[b]] for b in range(B)])
        assert torch.allclose(got, want, rtol=1e-3, atol=1e-4 * float(whole.abs().max())), k


def test_block_training_step():
    """Norm, convolution and scan forward and backward in a row, against autograd over the definitions."""
    r = gen(4)
    B, D, L, N, T = 2, 24, 70, 6, 4
    x, w, conv = r(B * L, D), 1 + 0.1 * r(D), r(D, T) / 2
    delta, bm, cm, A = r(B, D, L) - 3, r(B, 1, N, L), r(B, 1, N, L), -torch.rand(D, N, generator=torch.Generator().manual_seed(1)) - 0.2
    gy = r(B, D, L)
    v = leaves(x=x, w=w, conv=conv, A=A)
    s = R.rms_norm(v["x"], v["w"], 1e-6).view(B, L, D).transpose(1, 2)
    c, _ = R.short_conv(s, v["conv"], None, True)
    y, _ = R.selective_scan(c, R.up(delta), v["A"], R.up(bm), R.up(cm))
    (y * R.up(gy)).sum().backward()
    n = H.rms_norm(dev(x), dev(w))
    nt = n.view(B, L, D).transpose(1, 2).contiguous()
    u = H.short_conv(nt, dev(conv), silu=True)
    args = (u, dev(delta), dev(A), dev(bm), dev(cm))
    close(H.selective_scan(*args), y.detach(), 600, None, "y")
    g = H.selective_scan_backward(*args, dev(gy))
    gc, gconv, _, _ = H.short_conv_backward(nt, dev(conv), g["gu"], silu=True)
    gx, gw = H.rms_norm_backward(dev(x), dev(w), gc.transpose(1, 2).contiguous().view(B * L, D))
    for got, key, many in ((gx, "x", 1), (gw, "w", 4), (gconv, "conv", 4), (g["gA"], "A", 4)):
        # three operators' roundings in a row, sums over batch and time of terms of both signs
        close(got, v[key].grad, 2000 * many, None, key)


def every_call():
    """name -> (call into fixed buffers, the buffers it writes): each entry point at a small size."""
    t, r = torch.bfloat16, gen(11)
    B, D, L, N, T = 2, 40, 1200, 16, 4
    x, w, b = dev(r(B, D, L).to(t)), dev(r(D, T)), dev(r(D))
    a, _, _ = scan_inputs((B, D, 1, N, L, True, True, True, True, True, None), t, 1)
    on = scan_on_gpu(a, None, True)
    gy = dev(r(B, D, L).to(t))
    rows, wn = dev(r(300, 640).to(t)), dev(r(640))
    q, s = H.quantize(rows)
    wq, ws = H.quantize(dev(r(96, 640)), 128)
    flat = lambda v: [x for x in (v.values() if isinstance(v, dict) else v if isinstance(v, tuple) else (v,)) if x is not None]  # noqa: E731
    calls = {
        "short_conv": lambda: H.short_conv(x, w, b, silu=True, return_state=True),
        "short_conv_backward": lambda: H.short_conv_backward(x, w, gy, b, silu=True),
        "selective_scan": lambda: H.selective_scan(**on, return_state=True),
        "selective_scan_backward": lambda: H.selective_scan_backward(**on, gy=gy),
        "rms_norm": lambda: H.rms_norm(rows, wn, residual=rows),
        "rms_norm_quantized": lambda: H.rms_norm_quantized(rows, wn, residual=rows),
        "rms_norm_backward": lambda: H.rms_norm_backward(rows, wn, rows),
        "quantize": lambda: H.quantize(rows),
        "scaled_matmul": lambda: H.scaled_matmul(q, s, wq, ws),
        "scaled_matmul_rows": lambda: H.scaled_matmul(q[:5], s[:5], wq, ws, out_dtype=torch.float32),
    }
    return {k: (lambda f=f: flat(f())) for k, f in calls.items()}


def bits(ts):
    return [x.detach().view(torch.uint8).clone() for x in ts]


def test_calls_replay_from_graphs():
    """Each call captured and replayed several times, with eager work between, gives the eager bits."""
    for name, call in every_call().items():
        want = bits(call())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        for k in range(3):
            for o in out:
                o.view(torch.uint8).fill_(255)
            torch.randn(1 << 20, device=DEV).sum()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(bits(out), want)), (name, k)


def test_calls_on_two_streams_at_once():
    """The same calls on two streams, each with its own buffers, give the bits of one after the other."""
    calls = every_call()
    want = {k: bits(f()) for k, f in calls.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for st in streams:
        with torch.cuda.stream(st):
            got.append({k: f() for k, f in calls.items()})
    torch.cuda.synchronize()
    for g in got:
        for k in calls:
            assert all(torch.equal(a, b) for a, b in zip(bits(g[k]), want[k])), k


def test_steps_replay_from_a_graph():
    """A captured token: state and output move on with each replay as they do eagerly."""
    t, B, D, N, T = torch.bfloat16, 4, 48, 16, 4
    r = gen(12)
    x, w, cs0 = dev(r(B, D).to(t)), dev(r(D, T)), dev(r(B, D, T - 1).to(t))
    delta, z = dev(r(B, D).to(t)), dev(r(B, D).to(t))
    bm, cm, A, ss0 = dev(r(B, 1, N).to(t)), dev(r(B, 1, N).to(t)), dev(-torch.rand(D, N)), dev(r(B, D, N))

    def token(cs, ss, y):
        u = H.short_conv_step(x, w, cs, silu=True)
        return H.selective_scan_step(u, delta, A, bm, cm, ss, z=z, out=y)

    cs, ss, want = cs0.clone(), ss0.clone(), []
    for _ in range(4):
        want.append(token(cs, ss, torch.empty_like(x)).clone())
    gcs, gss, gy = cs0.clone(), ss0.clone(), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(cs0.clone(), ss0.clone(), gy)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        token(gcs, gss, gy)
    gcs.copy_(cs0)
    gss.copy_(ss0)
    for k in range(4):
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, want[k]), k
    assert torch.equal(gcs, cs) and torch.equal(gss, ss)


def test_offsets_beyond_32_bits():
    """The last rows of arrays of more than 2^31 values are what they are alone."""
    t, D, L = torch.bfloat16, 1030, 1 << 21
    x = torch.empty(1, D, L, dtype=t, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(3))
    assert x.numel() > 1 << 31
    r = gen(15)
    w = dev(r(D, 4))
    last = x[:, -2:].contiguous()
    y = H.short_conv(x, w, silu=True)
    assert torch.equal(y[:, -2:], H.short_conv(last, w[-2:].contiguous(), silu=True))
    del y
    gx, gw, _, _ = H.short_conv_backward(x, w, x, silu=True)
    gx2, gw2, _, _ = H.short_conv_backward(last, w[-2:].contiguous(), last, silu=True)
    assert torch.equal(gx[:, -2:], gx2)
    # the same products, in other partials: 2^21 terms of both signs, chains of 128 in a thread, then sums of those
    assert torch.allclose(gw[-2:], gw2, rtol=0, atol=200 * EPS32 * float(gw2.abs().max()) * 8)
    del gx
    N = 2
    bm, A = dev(r(1, 1, N, L).to(t)), dev(-torch.rand(D, N) - 0.1)
    y, h = H.selective_scan(x, x, A, bm, bm, return_state=True)
    y2, h2 = H.selective_scan(last, last, A[-2:].contiguous(), bm, bm, return_state=True)
    # segments of other lengths: the state's roundings, as in test_selective_scan, twice; time steps of about 1 here
    close(h[:, -2:], h2.cpu().double(), 2 * 416, float(h2.abs().max()) + 1, "state")
    off = (y[:, -2:].float() - y2.float()).abs().max()
    assert float(off) <= 2 * 2.0 ** -8 * float(y2.float().abs().max())
    del y
    rows = x.view(D * 16, L // 16)
    assert torch.equal(H.rms_norm(rows, dev(torch.ones(L // 16)))[-1], H.rms_norm(rows[-1:].contiguous(), dev(torch.ones(L // 16)))[0])
    q, s = H.quantize(rows)
    q2, s2 = H.quantize(rows[-1:].contiguous())
    assert torch.equal(q[-1].view(torch.uint8), q2[0].view(torch.uint8)) and torch.equal(s[-1], s2[0])


def test_a_workspace_of_the_callers():
    """A caller's workspace is used as it is, and one too small is refused."""
    t, r = torch.float32, gen(13)
    B, D, L, N = 1, 16, 2100, 4
    a, _, _ = scan_inputs((B, D, 1, N, L, True, True, True, True, True, None), t, 3)
    on = scan_on_gpu(a, None, True)
    need = H.selective_scan_workspace_bytes(B, D, N, L)
    assert need > 0
    want = H.selective_scan(**on)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(H.selective_scan(**on, workspace=ws), want)
    assert bool((ws[need:] == 255).all())
    for call, n in ((lambda w: H.selective_scan(**on, workspace=w), need),
                    (lambda w: H.selective_scan_backward(**on, gy=on["u"], workspace=w),
                     H.selective_scan_backward_workspace_bytes(B, D, 1, N, L)),
                    (lambda w: H.short_conv_backward(on["u"], dev(r(D, 4)), on["u"], workspace=w),
                     H.short_conv_backward_workspace_bytes(B, D, 4, L)),
                    (lambda w: H.rms_norm_backward(on["u"], dev(r(L)), on["u"], workspace=w),
                     H.rms_norm_backward_workspace_bytes(B * D, L))):
        with pytest.raises(H.HyenaError) as e:
            call(torch.empty(n - 1, dtype=torch.uint8, device=DEV))
        assert e.value.code == 5


def test_binding_refuses_what_does_not_fit():
    t, r = torch.float32, gen(14)
    x, w = dev(r(2, 8, 20)), dev(r(8, 4))
    with pytest.raises(ValueError):
        H.short_conv(x.transpose(1, 2), w)                                    # not contiguous
    with pytest.raises(ValueError):
        H.short_conv(x, w[:5].contiguous())                                   # another channel count
    with pytest.raises(TypeError):
        H.short_conv(x.half(), w)
    with pytest.raises(TypeError):
        H.short_conv(x, w, lengths=torch.tensor([1, 2], device=DEV))          # int64 lengths
    with pytest.raises(ValueError):
        H.short_conv(x, w, state=dev(r(2, 8, 2)))
    with pytest.raises(TypeError):
        H.short_conv(x, w.cpu())
    with pytest.raises(H.HyenaError) as e:
        H.short_conv(x, dev(r(8, 17)))
    assert e.value.code == 2
    with pytest.raises(H.HyenaError) as e:
        H.short_conv(x, w, out=x)
    assert e.value.code == 6
    with pytest.raises(H.HyenaError) as e:
        H.short_conv(x.view(-1)[1:9].view(1, 8, 1), w, out=dev(r(1, 8, 1)))
    assert e.value.code == 4
    on = scan_on_gpu(scan_inputs((1, 4, 1, 4, 6, True, True, True, True, True, None), t, 1)[0], None, True)
    with pytest.raises(ValueError):
        H.selective_scan(**dict(on, Bm=on["Bm"][..., :5].contiguous()))
    with pytest.raises(ValueError):
        H.selective_scan(**dict(on, z=on["z"].view(4, 6)))
    with pytest.raises(TypeError):
        H.selective_scan(**dict(on, state=on["state"].double()))
    with pytest.raises(ValueError):
        H.rms_norm(x, dev(r(19)))
    q, s = H.quantize(dev(r(4, 24)))
    wq, ws = H.quantize(dev(r(8, 24)), 128)
    with pytest.raises(H.HyenaError) as e:
        H.scaled_matmul(q, s, wq, ws)                                         # K is no multiple of 16
    assert e.value.code == 3
    q, s = H.quantize(dev(r(4, 32)))
    with pytest.raises(ValueError):
        H.scaled_matmul(q, s, wq, ws)
    with pytest.raises(TypeError):
        H.scaled_matmul(q, s, q.view(torch.uint8), s, out_dtype=torch.float32)
    with pytest.raises(TypeError):
        H.scaled_matmul(q, s, q, s, out_dtype=torch.float16)
