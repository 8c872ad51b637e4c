"""Refusals of the state-space block's Python entry points that need a GPU
tensor to get to."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests.test_ssm import dev, gen

pytestmark = pytest.mark.gpu


def calls():
    """name -> (function, its required arguments, those that are required tensors)"""
    r = gen(1)
    x, row, w, A, b = dev(r(2, 8, 20)), dev(r(2, 8)), dev(r(8, 4)), dev(-r(8, 4).abs()), dev(r(2, 1, 4, 20))
    q, s = H.quantize(dev(r(4, 32)))
    wq, ws = H.quantize(dev(r(8, 32)), 128)
    one = b[..., 0].contiguous()
    return {
        "short_conv": (H.short_conv, dict(x=x, w=w)),
        "short_conv_step": (H.short_conv_step, dict(x=row, w=w, state=dev(r(2, 8, 3)))),
        "short_conv_backward": (H.short_conv_backward, dict(x=x, w=w, gy=x)),
        "selective_scan": (H.selective_scan, dict(u=x, delta=x, A=A, Bm=b, Cm=b)),
        "selective_scan_step": (H.selective_scan_step, dict(u=row, delta=row, A=A, Bm=one, Cm=one, state=dev(r(2, 8, 4)))),
        "selective_scan_backward": (H.selective_scan_backward, dict(u=x, delta=x, A=A, Bm=b, Cm=b, gy=x)),
        "rms_norm": (H.rms_norm, dict(x=x, weight=dev(r(20)))),
        "rms_norm_quantized": (H.rms_norm_quantized, dict(x=x, weight=dev(r(20)))),
        "rms_norm_backward": (H.rms_norm_backward, dict(s=x, weight=dev(r(20)), gy=x)),
        "quantize": (H.quantize, dict(x=x)),
        "scaled_matmul": (H.scaled_matmul, dict(q=q, scales=s, wq=wq, wscales=ws)),
    }


def test_every_required_tensor_is_asked_for():
    """None, a list or a CPU tensor in a required place is a TypeError, or (None) the library's own refusal."""
    for name, (f, args) in calls().items():
        f(**args)
        for k, v in args.items():
            for bad in ([1.0], v.cpu()):
                with pytest.raises(TypeError):
                    f(**dict(args, **{k: bad}))
            with pytest.raises((TypeError, H.HyenaError)) as e:
                f(**dict(args, **{k: None}))
            assert e.type is TypeError or e.value.code == 1, (name, k)
