"""Linear attention at the most sequences and heads that a launch takes: more
than 2^22 of them, up to 2^24 workgroups."""
import os

import pytest
import torch

import hyena_long_conv_amd as H
from tests import linattn_reference as R
from tests.test_linattn import count, near
from tests.test_ssm import DEV


@pytest.mark.skipif(not os.path.exists(H.LIB_PATH), reason="library not built")
def test_sizes_of_launches():
    """Workgroups of 256 threads: one to a head of up to 64 columns, two up to 128, four beyond."""
    f, g = H.linear_attention_workspace_bytes, H.linear_attention_backward_workspace_bytes
    for Dv, most in ((64, 15), (128, 7), (256, 3)):
        assert f(1 << 20, 1, most, 8, Dv) == 0 and f(1 << 20, 1, most + 1, 8, Dv) == -1
        assert g(1 << 20, 1, most, most, most, most, Dv, 8) == 0 and g(1 << 20, 1, most + 1, most + 1, 1, 1, Dv, 8) == -1


@pytest.mark.gpu
def test_four_million_heads():
    """Over 2^22 sequences and heads: prompts of one token, their gradients, and a token."""
    B, N, D = 1 << 20, 5, 4
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, go = (torch.randn(B, 1, N, D, generator=g, device=DEV) for _ in range(4))
    state = torch.randn(B, N, D, D, generator=g, device=DEV)
    decay = -torch.rand(N, generator=g, device=DEV)
    ref = R.linear_attention(q, k, v, decay, state=state, go=go)
    o, last = H.linear_attention(q, k, v, decay, state=state, return_state=True)
    got = H.linear_attention_backward(q, k, v, go, decay, state=state)
    c = count(1, D, D)
    near(o, *ref["o"], c, 0, "o")
    near(last, *ref["state"], c, 0, "state")
    for name in ("gq", "gk", "gv", "gstate"):
        near(got[name], *ref[name], c + 8, 0, name)
    one = H.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], state, decay)
    near(one, ref["o"][0][:, 0], ref["o"][1][:, 0], 2 * D + 16, 0, "o of a token")
    near(state, *ref["state"], 16, 0, "state of a token")


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("heads,Dk,Dv", [((3, 1, 3), 128, 100), ((2, 2, 2), 64, 128), ((2, 1, 1), 40, 64)])
def test_backward_workspace_as_large_as_asked_for(heads, Dk, Dv, io):
    """One size serves both types, whose splits of the time axis differ; nothing behind it is written."""
    L, N = 5000, max(heads)
    g = torch.Generator(device=DEV).manual_seed(2)
    t = torch.bfloat16 if io == "bf16" else torch.float32
    q, k, v, go = (torch.randn(1, L, h, d, generator=g, device=DEV).to(t) for h, d in ((heads[0], Dk), (heads[1], Dk), (heads[2], Dv), (N, Dv)))
    need = H.linear_attention_backward_workspace_bytes(1, L, N, *heads, Dk, Dv)
    room = torch.full((need + 4096,), 85, dtype=torch.uint8, device=DEV)
    want = H.linear_attention_backward(q, k, v, go)
    got = H.linear_attention_backward(q, k, v, go, workspace=room[:need])
    for name in ("gq", "gk", "gv"):
        assert torch.equal(got[name], want[name]), name
    assert bool((room[need:] == 85).all())
