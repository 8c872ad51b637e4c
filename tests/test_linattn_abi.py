"""Host-side checks of the linear-attention block's entry points: bad arguments
come back as a status before anything touches a GPU, and the helper functions
that need none.  Runs on the CPU, also against the library's sanitized host
build."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import hyena_long_conv_amd as H
from hyena_long_conv_amd import linattn
from tests import linattn_reference as R
from tests.test_ssm_abi import ALIAS, ALIGN, BIG, NULL, SHAPE, UNSUP, WS, P

pytestmark = pytest.mark.skipif(not os.path.exists(H.LIB_PATH), reason="library not built")
vp = ctypes.c_void_p
ATTENTION = ["hyena_linear_attention", "hyena_linear_attention_step", "hyena_linear_attention_backward"]


def attention(which, io=0, o=P[10], so=0, ws=P[11], wsb=BIG, null=False, **k):
    B, L, N = k.get("B", 2), k.get("L", 64), k.get("H", 4)
    Hq, Hk, Hv, Dk, Dv = k.get("Hq", 4), k.get("Hk", 2), k.get("Hv", 2), k.get("Dk", 32), k.get("Dv", 16)
    dense = lambda h, d: (L * h * d, h * d, d)  # noqa: E731
    p = linattn.LinearAttentionParams(
        B, L, N, Hq, Hk, Hv, Dk, Dv, k.get("scale", 1.0), 0, k.get("q", P[0]), k.get("k", P[1]), k.get("v", P[2]),
        *k.get("qs", dense(Hq, Dk)), *k.get("ks", dense(Hk, Dk)), *k.get("vs", dense(Hv, Dv)), k.get("decay", P[3]),
        k.get("state", 0), k.get("lengths", 0))
    pp, f = None if null else ctypes.byref(p), getattr(H.lib(), which)
    if which == "hyena_linear_attention_step":
        return f(pp, vp(k.get("st", P[12])), vp(o), io, None)
    if which == "hyena_linear_attention_backward":
        g = linattn.LinearAttentionGrads(k.get("gq", P[20]), k.get("gk", P[21]), k.get("gv", P[22]), k.get("gs", 0))
        return f(pp, vp(k.get("go", P[13])), vp(k.get("gso", 0)), None if k.get("nog") else ctypes.byref(g), io, vp(ws), wsb, None)
    return f(pp, vp(o), vp(so), io, vp(ws), wsb, None)


@pytest.mark.parametrize("which", ATTENTION)
def test_linear_attention_rejects_bad_arguments(which):
    c = lambda **k: attention(which, **k)  # noqa: E731
    assert c(null=True) == NULL and c(q=0) == NULL and c(k=0) == NULL and c(v=0) == NULL
    assert c(B=0) == SHAPE and c(H=0) == SHAPE and c(Hq=3) == SHAPE and c(Hk=8) == SHAPE and c(Hv=0) == SHAPE
    assert c(Dk=0) == SHAPE and c(Dk=257) == SHAPE and c(Dv=0) == SHAPE and c(Dv=257) == SHAPE
    assert c(B=1 << 20, H=1 << 12, Hq=1, Hk=1, Hv=1) == SHAPE
    assert c(qs=(-1, 1, 1)) == SHAPE and c(ks=(0, (1 << 38) + 1, 0)) == SHAPE and c(vs=(0, 0, -8)) == SHAPE
    assert c(io=2) == UNSUP and c(scale=float("nan")) == UNSUP and c(scale=float("inf")) == UNSUP
    assert c(q=P[0] + 2) == ALIGN and c(decay=P[3] + 2) == ALIGN and c(v=P[2] + 1, io=1) == ALIGN
    if which != "hyena_linear_attention_step":
        assert c(L=0) == SHAPE and c(L=(1 << 22) + 1) == SHAPE
        assert c(state=P[30] + 4) == ALIGN and c(lengths=P[30] + 2) == ALIGN
        assert c(B=1 << 20, H=16, L=1) == UNSUP
    if which != "hyena_linear_attention_backward":
        assert c(o=0) == NULL and c(o=P[10] + 8) == ALIGN and c(o=P[2]) == ALIAS and c(o=P[1] + 64) == ALIAS
        # a view's last values, far from its first
        far = (1 << 30, 1 << 20, 1 << 12)
        end = ((1 << 30) + 63 * (1 << 20) + (1 << 12) + 16) * 4
        more = dict(L=64) if which == "hyena_linear_attention" else {}
        if more:
            assert c(vs=far, o=P[2] + end - 16, **more) == ALIAS
    if which == "hyena_linear_attention":
        need = H.linear_attention_workspace_bytes(2, 4096, 4, 32, 16)
        assert need > 0 and H.linear_attention_workspace_bytes(2, 64, 4, 32, 16) == 0
        assert c(L=4096, ws=0) == WS and c(L=4096, wsb=need - 1) == WS and c(L=4096, ws=P[0]) == ALIAS and c(L=4096, ws=P[11] + 4) == ALIGN
        assert c(so=P[14], state=P[14]) == ALIAS and c(so=P[10]) == ALIAS and c(so=P[14] + 8) == ALIGN
    if which == "hyena_linear_attention_step":
        assert c(st=0) == NULL and c(st=P[12] + 4) == ALIGN and c(st=P[0]) == ALIAS and c(st=P[10]) == ALIAS
        assert c(B=1 << 20, H=16, Hq=16, Hk=16, Hv=16) == UNSUP
    if which == "hyena_linear_attention_backward":
        for k in ("gq", "gk", "gv", "go"):
            assert c(**{k: 0}) == NULL, k
            assert c(**{k: P[31] + 8}) == ALIGN, k
        assert c(nog=True) == NULL
        need = H.linear_attention_backward_workspace_bytes(2, 64, 4, 4, 2, 2, 32, 16)
        assert need == 2 * 64 * 4 * (32 + 16) * 4       # fp32 gradients of k and v for each head, which share two
        assert H.linear_attention_backward_workspace_bytes(2, 64, 4, 4, 4, 4, 32, 16) == 0
        assert c(wsb=need - 1) == WS and c(ws=0) == WS and c(ws=P[1]) == ALIAS
        assert c(gq=P[0]) == ALIAS and c(gk=P[13]) == ALIAS and c(gv=P[20]) == ALIAS and c(gs=P[21]) == ALIAS
        assert c(gs=P[14], state=P[14]) == ALIAS and c(gs=P[14], gso=P[14]) == ALIAS


def test_workspace_sizes_refuse_what_the_calls_refuse():
    f, g, n = H.linear_attention_workspace_bytes, H.linear_attention_backward_workspace_bytes, H.group_norm_backward_workspace_bytes
    assert f(0, 1, 1, 1, 1) == -1 and f(1, 0, 1, 1, 1) == -1 and f(1, 1, 1, 257, 1) == -1 and f(1, 1, 1, 1, 0) == -1
    assert g(1, 1, 4, 3, 4, 4, 1, 1) == -1 and g(1, 1, 4, 4, 8, 4, 1, 1) == -1
    assert n(0, 8, 1) == -1 and n(4, 8, 3) == -1 and n(4, 8, 0) == -1 and n(4, 8, 2) > 0
    # the states between segments of the longest sequence, and nothing where heads alone fill the chip
    assert 0 < f(1, 1 << 22, 1, 256, 256) <= 256 * 256 * 256 * 4 and f(64, 4096, 64, 64, 64) == 0


def test_workspace_sizes_of_calls_too_large_to_launch():
    """Sizes whose launches a call refuses (UNSUPPORTED): -1, where sums of their bytes pass 63 bits too."""
    f, g, n = H.linear_attention_workspace_bytes, H.linear_attention_backward_workspace_bytes, H.group_norm_backward_workspace_bytes
    for heads in ((1, 1, 1), (1, 1, 1024), (1024, 1024, 1024)):
        assert g(1 << 20, 1 << 22, 1024, *heads, 256, 256) == -1
    assert f(1 << 20, 1 << 22, 1024, 256, 256) == -1 and f(1 << 20, 1, 16, 16, 16) == -1
    assert attention("hyena_linear_attention", B=1 << 20, H=16, L=1, Dk=16, Dv=16) == UNSUP
    assert attention("hyena_linear_attention_backward", B=1 << 20, H=1024, L=1 << 22, Hq=1, Hk=1, Hv=1, Dk=256, Dv=256) == UNSUP
    assert n(1 << 24, 10000, 1) == -1 and norm(back=True, rows=1 << 24, D=10000, G=1) == UNSUP
    assert n((1 << 24) - 1, 10000, 1) > 0


def rotary(x=P[0], out=P[1], io=0, null=False, **k):
    B, L, N, D = k.get("B", 2), k.get("L", 8), k.get("H", 4), k.get("D", 64)
    p = linattn.RotaryParams(B, L, N, D, k.get("R", 32), k.get("il", 0), k.get("inv", 0), k.get("scale", 1.0),
                             *k.get("xs", (L * N * D, N * D, D)), k.get("freq", P[2]), k.get("pos", 0), *k.get("ps", (0, 1)))
    return H.lib().hyena_rotary(None if null else ctypes.byref(p), vp(x), vp(out), io, None)


def test_rotary_rejects_bad_arguments():
    c = rotary
    assert c(null=True) == NULL and c(x=0) == NULL and c(out=0) == NULL and c(freq=0) == NULL
    assert c(B=0) == SHAPE and c(L=0) == SHAPE and c(H=0) == SHAPE and c(D=1, R=2) == SHAPE and c(D=(1 << 16) + 1) == SHAPE
    assert c(R=0) == SHAPE and c(R=33) == SHAPE and c(R=66) == SHAPE
    assert c(xs=(0, -1, 0)) == SHAPE and c(pos=P[3], ps=(-1, 0)) == SHAPE
    assert c(il=2) == UNSUP and c(inv=2) == UNSUP and c(io=2) == UNSUP and c(scale=float("nan")) == UNSUP
    assert c(B=1 << 15, L=1 << 15, H=1, D=1 << 10, R=1 << 10) == UNSUP
    assert c(out=P[1] + 8) == ALIGN and c(freq=P[2] + 4) == ALIGN and c(pos=P[3] + 2) == ALIGN and c(x=P[0] + 1, io=1) == ALIGN
    assert c(out=P[0] + 16) == ALIAS and c(out=P[2]) == ALIAS and c(pos=P[1]) == ALIAS
    # in place: heads have to lie apart
    assert c(out=P[0], xs=(0, 256, 64)) == ALIAS and c(out=P[0], xs=(2048, 255, 64)) == ALIAS
    assert c(out=P[0], xs=(2048, 256, 63)) == ALIAS and c(out=P[0], xs=(2048, 64, 500)) == ALIAS


def norm(y=P[1], io=0, back=False, null=False, **k):
    p = linattn.GroupNormParams(k.get("rows", 4), k.get("D", 256), k.get("G", 4), k.get("silu", 0), k.get("eps", 1e-5),
                                k.get("x", P[0]), k.get("z", 0), k.get("w", P[2]), k.get("b", P[3]))
    pp = None if null else ctypes.byref(p)
    if back:
        return H.lib().hyena_group_norm_backward(pp, vp(k.get("gy", P[4])), vp(y), vp(k.get("gw", P[5])), vp(k.get("gb", P[6])),
                                                 vp(k.get("gz", 0)), io, vp(k.get("ws", P[7])), k.get("wsb", BIG), None)
    return H.lib().hyena_group_norm(pp, vp(y), io, None)


@pytest.mark.parametrize("back", [False, True])
def test_group_norm_rejects_bad_arguments(back):
    c = lambda **k: norm(back=back, **k)  # noqa: E731
    assert c(null=True) == NULL and c(x=0) == NULL and c(y=0) == NULL
    assert c(rows=0) == SHAPE and c(D=0) == SHAPE and c(G=0) == SHAPE and c(G=3) == SHAPE and c(D=1 << 21) == SHAPE
    assert c(rows=(1 << 31) + 1) == SHAPE
    z = dict(z=P[8], **(dict(gz=P[9]) if back else {}))
    assert c(silu=2) == UNSUP and c(silu=1, **z) == UNSUP and c(io=2) == UNSUP
    assert c(eps=-1.0) == UNSUP and c(eps=float("nan")) == UNSUP and c(eps=float("inf")) == UNSUP
    assert c(rows=1 << 24, D=10000, G=1) == UNSUP
    assert c(x=P[0] + 8) == ALIGN and c(y=P[1] + 4) == ALIGN and c(w=P[2] + 1) == ALIGN
    assert c(y=P[0]) == ALIAS and c(y=P[2]) == ALIAS
    if back:
        assert c(gy=0) == NULL and c(z=P[8]) == NULL and c(gz=P[9]) == NULL
        need = H.group_norm_backward_workspace_bytes(4, 256, 4)
        assert c(wsb=need - 1) == WS and c(ws=0) == WS and c(ws=P[0]) == ALIAS
        assert c(gw=P[4]) == ALIAS and c(gb=P[5]) == ALIAS and c(z=P[8], gz=P[8]) == ALIAS


# ---------------------------------------------------- what needs no library

def test_rotary_frequencies():
    f = lambda *a, **k: H.rotary_frequencies(*a, device="cpu", **k)  # noqa: E731
    plain, one = f(8)
    assert plain.dtype == torch.float64 and one == 1.0
    assert torch.allclose(plain, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-12)
    assert torch.equal(f(8, scaling="linear", factor=4.0)[0], plain / 4)
    ntk = f(8, scaling="ntk", factor=4.0)[0]
    assert float(ntk[0]) == 1.0 and math.isclose(float(ntk[-1]), float(plain[-1]) / 4, rel_tol=1e-12)
    wide, _ = f(64)
    y, s = f(64, scaling="yarn", factor=8.0, context=2048)
    turns = 2048 * wide / (2 * math.pi)
    assert math.isclose(s, 0.1 * math.log(8.0) + 1)
    assert torch.equal(y[turns >= 32], wide[turns >= 32]) and torch.allclose(y[turns <= 1], wide[turns <= 1] / 8, rtol=1e-12)
    between = (turns > 1) & (turns < 32)
    assert bool(((y < wide) & (y > wide / 8))[between].all()) and bool(between.any())
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, scaling="cubic"), dict(dim=8, factor=0.5), dict(dim=2, scaling="ntk"),
                dict(dim=8, base=0.0), dict(dim=8, scaling="yarn", turns=(2.0, 2.0)), dict(dim=8, factor=float("inf"))):
        with pytest.raises(ValueError):
            f(**bad)


def test_definitions_agree():
    """The recurrence and the double sum over pairs of tokens, and their gradients."""
    g = torch.Generator().manual_seed(1)
    r = lambda *n: torch.randn(*n, generator=g, dtype=torch.float64)  # noqa: E731
    B, L, N, Dk, Dv = 3, 11, 2, 4, 5
    a = dict(q=r(B, L, N, Dk), k=r(B, L, N, Dk), v=r(B, L, N, Dv), state=r(B, N, Dk, Dv))
    decay, lengths, go, gso = -r(N).abs(), torch.tensor([11, 0, 6]), r(B, L, N, Dv), r(B, N, Dk, Dv)
    v = {k: x.clone().requires_grad_() for k, x in a.items()}
    o, s = R.linear_attention_by_sums(v["q"], v["k"], v["v"], decay, 0.7, v["state"], lengths)
    ((o * go).sum() + (s * gso).sum()).backward()
    got = R.linear_attention(**a, log_decay=decay, scale=0.7, lengths=lengths, go=go, gstate_out=gso)
    want = dict(o=o.detach(), state=s.detach(), gq=v["q"].grad, gk=v["k"].grad, gv=v["v"].grad, gstate=v["state"].grad)
    for k, w in want.items():
        assert torch.allclose(got[k][0], w, rtol=1e-12, atol=1e-13), k
        assert bool((got[k][1] >= w.abs() - 1e-12).all()), k


def test_binding_needs_gpu_tensors():
    x = torch.zeros(1, 4, 2, 8)
    for call in (lambda: H.linear_attention(x, x, x), lambda: H.linear_attention_step(x[0], x[0], x[0], x),
                 lambda: H.linear_attention_backward(x, x, x, x), lambda: H.rotary(x, torch.zeros(4)), lambda: H.group_norm(x, 2),
                 lambda: H.group_norm_backward(x, 2, x)):
        with pytest.raises(TypeError):
            call()


def test_under_sanitizers():
    """The checks above against the host build with AddressSanitizer and UndefinedBehaviorSanitizer."""
    if os.environ.get("HYENA_LIB"):
        pytest.skip("already in the sanitized run")
    from hyena_long_conv_amd.build import BUILD, build_hostcheck
    from tests.test_hostcheck import ROOT, _runtime
    lib = build_hostcheck(os.path.join(BUILD, "libhyena_hostcheck_linattn.so"))
    env = dict(os.environ, HYENA_LIB=lib, LD_PRELOAD=f"{_runtime('libasan.so')}:{_runtime('libubsan.so')}",
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.join("tests", "test_linattn_abi.py")],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0 and "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out
