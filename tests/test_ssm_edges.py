"""The state-space block's operators where a value is not finite, a sequence
is empty or a limit is near: what such a value may reach, and what stays the
bits of a call without it."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests import ssm_reference as R
from tests.test_ssm import TYPES, close, dev, gen, leaves

pytestmark = pytest.mark.gpu


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
