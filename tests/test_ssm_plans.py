"""The launches that the cases of tests/test_ssm_wide.py are there for, from
the rules in csrc/ssm.hpp compiled for the host, and the float64 definition
those cases are compared with.  Runs on the CPU."""
import os
import shutil
import subprocess

import pytest
import torch

from tests import ssm_reference as R
from tests.test_ssm_wide import CONV, SCAN

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("ssm_plan") / "ssm_plan_host")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I",
                        os.path.join(ROOT, "hyena_long_conv_amd", "csrc"), os.path.join(ROOT, "tests", "ssm_plan_host.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(*args):
        words = subprocess.check_output([exe, *map(str, args)], text=True).split()
        return dict(zip(words[::2], map(int, words[1::2])))
    return ask


@pytest.mark.parametrize("name", SCAN)
def test_scan_cases_have_their_launches(plan, name):
    sizes, want = SCAN[name]
    got = plan("scan", *sizes)
    assert {k: got[k] for k in want} == want, got


@pytest.mark.parametrize("name", CONV)
def test_conv_cases_have_their_walks(plan, name):
    sizes, walks = CONV[name]
    assert plan("conv", *sizes)["walks"] == walks


@pytest.mark.parametrize("softplus", [True, False])
def test_definition_with_sizes_agrees_with_autograd(softplus):
    g = torch.Generator().manual_seed(7)
    r = lambda *n: torch.randn(*n, generator=g, dtype=torch.float64)  # noqa: E731
    B, D, G, N, L = 3, 6, 2, 4, 11
    a = dict(u=r(B, D, L), delta=r(B, D, L) if softplus else r(B, D, L).abs() * 0.1, A=-r(D, N).abs(), Bm=r(B, G, N, L),
             Cm=r(B, G, N, L), skip=r(D), z=r(B, D, L), delta_bias=r(D) if softplus else r(D).abs() * 0.1, state=r(B, D, N))
    lengths = torch.tensor([11, 0, 5], dtype=torch.int32)
    gy, gso = r(B, D, L), r(B, D, N)
    v = {k: t.clone().requires_grad_(True) for k, t in a.items()}
    y, h = R.selective_scan(*[v[k] for k in ("u", "delta", "A", "Bm", "Cm", "skip", "z", "delta_bias")], softplus, v["state"],
                            lengths)
    (y * gy).sum().add((h * gso).sum()).backward()
    got = R.selective_scan_with_sizes(**a, softplus=softplus, lengths=lengths, gy=gy, gstate_out=gso)
    want = dict(y=y.detach(), h=h.detach(), gu=v["u"].grad, gdelta=v["delta"].grad, gA=v["A"].grad, gB=v["Bm"].grad,
                gC=v["Cm"].grad, gskip=v["skip"].grad, gz=v["z"].grad, gdelta_bias=v["delta_bias"].grad, gstate=v["state"].grad)
    assert set(got) == set(want)
    for k, (value, size) in got.items():
        assert torch.allclose(value, want[k], rtol=1e-11, atol=1e-12), k
        assert bool((size >= value.abs() - 1e-12).all()), k
