"""Host-side checks of the state-space block's entry points: bad arguments
come back as a status before anything touches a GPU.  Runs on the CPU, also
against the library's sanitized host build."""
import ctypes
import os
import subprocess
import sys

import pytest

import hyena_long_conv_amd as H
from hyena_long_conv_amd import ssm

pytestmark = pytest.mark.skipif(not os.path.exists(H.LIB_PATH), reason="library not built")

OK, NULL, SHAPE, UNSUP, ALIGN, WS, ALIAS, HIP = range(8)
vp = ctypes.c_void_p
P = [0x1000000000 * k for k in range(1, 40)]          # well-apart, aligned addresses that no call below touches
BIG = 1 << 40


def conv(x=P[0], y=P[1], so=0, io=0, which="hyena_short_conv", **k):
    p = ssm.ShortConvParams(k.get("B", 2), k.get("L", 64), k.get("D", 8), k.get("T", 4), k.get("silu", 1), 0,
                            k.get("w", P[2]), k.get("bias", 0), k.get("state", 0), k.get("lengths", 0))
    f = getattr(H.lib(), which)
    if which == "hyena_short_conv_step":
        return f(vp(x), ctypes.byref(p), vp(so), vp(y), io, None)
    if which == "hyena_short_conv_backward":
        return f(vp(x), ctypes.byref(p), vp(k.get("gy", P[5])), vp(k.get("gso", 0)), vp(y), vp(k.get("gw", P[6])),
                 vp(k.get("gb", 0)), vp(k.get("gs", 0)), io, vp(k.get("ws", P[7])), k.get("wsb", BIG), None)
    return f(vp(x), ctypes.byref(p), vp(y), vp(so), io, None)


@pytest.mark.parametrize("which", ["hyena_short_conv", "hyena_short_conv_step", "hyena_short_conv_backward"])
def test_short_conv_rejects_bad_arguments(which):
    so = P[4] if which == "hyena_short_conv_step" else 0
    c = lambda **k: conv(which=which, **{"so": so, **k})  # noqa: E731
    assert c(x=0) == NULL
    assert c(y=0) == NULL
    assert c(w=0) == NULL
    assert c(B=0) == SHAPE and c(D=0) == SHAPE and c(D=-4) == SHAPE
    assert c(B=1 << 20, D=1 << 20) == SHAPE
    assert c(T=0) == SHAPE and c(T=17) == SHAPE
    assert c(silu=2) == UNSUP
    assert c(io=2) == UNSUP
    assert c(x=P[0] + 8) == ALIGN and c(y=P[1] + 2) == ALIGN and c(w=P[2] + 2) == ALIGN
    assert c(y=P[0]) == ALIAS and c(y=P[2]) == ALIAS
    if which != "hyena_short_conv_step":
        assert c(L=0) == SHAPE and c(L=(1 << 22) + 1) == SHAPE
        assert c(T=1, state=P[3]) == SHAPE
        assert c(state=P[3], y=P[3] + 16) == ALIAS
        assert c(lengths=P[3] + 2) == ALIGN
        assert c(B=1 << 10, D=1 << 20, L=1 << 20) == UNSUP      # more workgroups than a launch holds
    if which == "hyena_short_conv":
        assert c(so=P[3], state=P[3]) == ALIAS and c(so=P[1]) == ALIAS and c(T=1, so=P[4]) == SHAPE
    if which == "hyena_short_conv_step":
        assert c(so=0) == NULL and c(T=1) == SHAPE and c(so=P[0]) == ALIAS and c(so=P[4] + 4) == ALIGN
    if which == "hyena_short_conv_backward":
        assert c(gy=0) == NULL and c(gw=0) == NULL and c(ws=0) == NULL
        assert c(wsb=H.short_conv_backward_workspace_bytes(2, 8, 4, 64) - 1) == WS
        assert c(gw=P[5]) == ALIAS and c(gb=P[6]) == ALIAS and c(ws=P[0]) == ALIAS
        assert c(T=1, gs=P[8]) == SHAPE


def scan(io=0, which="hyena_selective_scan", y=P[10], so=0, ws=0, wsb=0, null=False, **k):
    p = ssm.SelectiveScanParams(k.get("B", 2), k.get("L", 64), k.get("D", 8), k.get("G", 2), k.get("N", 16),
                                k.get("softplus", 1), k.get("u", P[0]), k.get("delta", P[1]), k.get("A", P[2]),
                                k.get("Bm", P[3]), k.get("Cm", P[4]), k.get("skip", 0), k.get("z", 0),
                                k.get("bias", 0), k.get("state", 0), k.get("lengths", 0))
    pp = None if null else ctypes.byref(p)
    f = getattr(H.lib(), which)
    if which == "hyena_selective_scan_step":
        return f(pp, vp(so), vp(y), io, None)
    if which == "hyena_selective_scan_backward":
        g = ssm.SelectiveScanGrads(*[k.get(n, d) for n, d in (("gu", P[20]), ("gdelta", P[21]), ("gA", P[22]), ("gB", P[23]),
                                                              ("gC", P[24]), ("gskip", 0), ("gz", 0), ("gdb", 0), ("gs", 0))])
        return f(pp, vp(k.get("gy", P[11])), vp(k.get("gso", 0)), None if k.get("nog") else ctypes.byref(g), io, vp(ws),
                 wsb, None)
    return f(pp, vp(y), vp(so), io, vp(ws), wsb, None)


@pytest.mark.parametrize("which", ["hyena_selective_scan", "hyena_selective_scan_step", "hyena_selective_scan_backward"])
def test_selective_scan_rejects_bad_arguments(which):
    more = {"hyena_selective_scan_step": dict(so=P[12]), "hyena_selective_scan_backward": dict(ws=P[13], wsb=BIG)}.get(which, {})
    c = lambda **k: scan(which=which, **{**more, **k})  # noqa: E731
    assert c(null=True) == NULL
    for k in ("u", "delta", "A", "Bm", "Cm"):
        assert c(**{k: 0}) == NULL, k
    assert c(B=0) == SHAPE and c(D=0) == SHAPE and c(N=0) == SHAPE and c(N=65) == SHAPE
    assert c(G=0) == SHAPE and c(G=3) == SHAPE and c(G=16) == SHAPE
    assert c(softplus=3) == UNSUP and c(io=9) == UNSUP
    for k in ("u", "delta", "Bm", "Cm"):
        assert c(**{k: P[30] + 8}) == ALIGN, k
    assert c(skip=P[30] + 1) == ALIGN
    if which != "hyena_selective_scan_step":
        assert c(L=0) == SHAPE and c(L=(1 << 22) + 1) == SHAPE
        assert c(state=P[30] + 4) == ALIGN
    if which == "hyena_selective_scan":
        assert c(y=0) == NULL and c(y=P[0]) == ALIAS and c(y=P[3] + 16) == ALIAS and c(so=P[10]) == ALIAS
        assert c(so=P[14], state=P[14]) == ALIAS
        need = H.selective_scan_workspace_bytes(2, 8, 16, 4096)
        assert need > 0 and H.selective_scan_workspace_bytes(2, 8, 16, 64) == 0
        assert c(L=4096) == WS and c(L=4096, ws=P[15], wsb=need - 1) == WS
        assert c(L=4096, ws=P[0], wsb=need) == ALIAS and c(L=4096, ws=P[15] + 4, wsb=need) == ALIGN
    if which == "hyena_selective_scan_step":
        assert c(so=0) == NULL and c(y=0) == NULL and c(A=P[2] + 4) == ALIGN and c(so=P[3]) == ALIAS
    if which == "hyena_selective_scan_backward":
        for k in ("gu", "gdelta", "gA", "gB", "gC", "gy"):
            assert c(**{k: 0}) == NULL, k
        assert c(nog=True) == NULL and c(ws=0) == NULL
        assert c(z=P[5]) == NULL and c(gz=P[25]) == NULL         # gz goes with z
        need = H.selective_scan_backward_workspace_bytes(2, 8, 2, 16, 64)
        assert c(wsb=need - 1) == WS
        assert c(gu=P[0]) == ALIAS and c(gB=P[24]) == ALIAS and c(gs=P[22]) == ALIAS and c(ws=P[11]) == ALIAS
        assert c(B=1 << 15, L=1 << 20) == UNSUP
    assert H.selective_scan_workspace_bytes(2, 8, 65, 64) == -1
    assert H.selective_scan_backward_workspace_bytes(2, 8, 3, 16, 64) == -1


def test_norm_rejects_bad_arguments():
    lib = H.lib()
    f = lambda x=P[0], r=0, w=P[1], y=P[2], s=0, rows=4, D=256, eps=1e-6, io=0: lib.hyena_rms_norm(  # noqa: E731
        vp(x), vp(r), vp(w), vp(y), vp(s), rows, D, eps, io, None)
    assert f(x=0) == NULL and f(w=0) == NULL and f(y=0) == NULL
    assert f(r=P[3]) == NULL and f(s=P[3]) == NULL               # the residual goes with the sum's place
    assert f(rows=0) == SHAPE and f(D=0) == SHAPE and f(D=(1 << 20) + 1) == SHAPE and f(rows=(1 << 31) + 1) == SHAPE
    assert f(eps=-1.0) == UNSUP and f(eps=float("nan")) == UNSUP and f(eps=float("inf")) == UNSUP and f(io=4) == UNSUP
    assert f(rows=1 << 27) == UNSUP
    assert f(x=P[0] + 8) == ALIGN and f(y=P[2] + 4) == ALIGN
    assert f(y=P[0]) == ALIAS and f(r=P[3], s=P[3]) == ALIAS and f(r=P[3], s=P[2] + 16) == ALIAS
    g = lambda q=P[4], sc=P[5], y=P[2]: lib.hyena_rms_norm_quantized(  # noqa: E731
        vp(P[0]), None, vp(P[1]), vp(q), vp(sc), None, 4, 256, 1e-6, 0, None)
    assert g(q=0) == NULL and g(sc=0) == NULL and g(q=P[0]) == ALIAS and g(sc=P[4] + 16) == ALIAS
    need = H.rms_norm_backward_workspace_bytes(4, 256)
    assert H.rms_norm_backward_workspace_bytes(0, 256) == -1
    b = lambda s=P[0], w=P[1], gy=P[2], gs=0, gx=P[4], gw=P[5], ws=P[6], wsb=need: lib.hyena_rms_norm_backward(  # noqa: E731
        vp(s), vp(w), vp(gy), vp(gs), vp(gx), vp(gw), 4, 256, 1e-6, 0, vp(ws), wsb, None)
    assert b(s=0) == NULL and b(w=0) == NULL and b(gy=0) == NULL and b(gx=0) == NULL and b(gw=0) == NULL and b(ws=0) == NULL
    assert b(wsb=need - 1) == WS and b(gx=P[2]) == ALIAS and b(gs=P[4]) == ALIAS and b(gs=P[7] + 4) == ALIGN


def test_product_rejects_bad_arguments():
    lib = H.lib()
    f = lambda q=P[0], s=P[1], wq=P[2], ws=P[3], b=0, o=P[4], B=2, L=8, N=32, K=256, cm=0, io=1: lib.hyena_scaled_matmul(  # noqa: E731
        vp(q), vp(s), vp(wq), vp(ws), vp(b), vp(o), B, L, N, K, cm, io, None)
    assert f(q=0) == NULL and f(s=0) == NULL and f(wq=0) == NULL and f(ws=0) == NULL and f(o=0) == NULL
    assert f(B=0) == SHAPE and f(L=0) == SHAPE and f(N=0) == SHAPE and f(K=0) == SHAPE and f(N=(1 << 20) + 1) == SHAPE
    assert f(K=24) == UNSUP and f(cm=2) == UNSUP and f(io=3) == UNSUP
    assert f(q=P[0] + 8) == ALIGN and f(wq=P[2] + 1) == ALIGN and f(o=P[4] + 8) == ALIGN and f(b=P[5] + 2) == ALIGN
    assert f(o=P[0]) == ALIAS and f(o=P[2] + 16) == ALIAS
    g = lambda x=P[0], q=P[1], s=P[2], rows=4, K=100, br=1, io=0: lib.hyena_quantize(  # noqa: E731
        vp(x), vp(q), vp(s), rows, K, br, io, None)
    assert g(x=0) == NULL and g(q=0) == NULL and g(s=0) == NULL
    assert g(rows=0) == SHAPE and g(K=0) == SHAPE and g(br=2) == UNSUP and g(io=2) == UNSUP
    assert g(q=P[0]) == ALIAS and g(x=P[0] + 4) == ALIGN


def test_binding_needs_gpu_tensors():
    import torch
    x = torch.zeros(1, 4, 8)
    for call in (lambda: H.short_conv(x, torch.zeros(4, 4)), lambda: H.rms_norm(x, torch.ones(8)), lambda: H.quantize(x[0]),
                 lambda: H.selective_scan(x, x, torch.zeros(4, 4), x, x)):
        with pytest.raises(TypeError):
            call()


def test_under_sanitizers():
    """The checks above against the host build with AddressSanitizer and UndefinedBehaviorSanitizer."""
    if os.environ.get("HYENA_LIB"):
        pytest.skip("already in the sanitized run")
    from hyena_long_conv_amd.build import BUILD, build_hostcheck
    from tests.test_hostcheck import ROOT, _runtime
    lib = build_hostcheck(os.path.join(BUILD, "libhyena_hostcheck_ssm.so"))
    env = dict(os.environ, HYENA_LIB=lib, LD_PRELOAD=f"{_runtime('libasan.so')}:{_runtime('libubsan.so')}",
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.join("tests", "test_ssm_abi.py")],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0 and "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out
