"""The series of the scan's softplus: the coefficients that the device code
holds, against artanh in float64.  Runs on the CPU."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hyena_long_conv_amd", "csrc",
                      "ssm_device.hpp")


def test_series_within_its_stated_bound():
    body = open(SOURCE).read().split("float softplus_f(float x)")[1]
    first = re.search(r"float p = ([0-9.]+)f;", body)
    rest = re.findall(r"p = fmaf\(p, q, ([0-9.]+)f\);", body)
    c = [float(np.float32(v)) for v in (first.group(1), *rest)]
    assert len(c) == 4
    q = np.linspace(1e-3, 1 / 9, 200_001)             # s^2 for every e^-|x| in (0, 1]
    s = np.sqrt(q)
    p = np.polyval(c, q)
    # log1p(e) = 2 s (1 + q p): what p's error does to the relative error
    assert np.abs(q * p - (np.arctanh(s) / s - 1)).max() <= 1.7e-8
    q = np.linspace(0, 1e-3, 1001)                    # near 0 the series itself, its next term below 1e-10
    assert np.abs(q * np.polyval(c, q) - q * (1 / 3 + q * (1 / 5 + q * (1 / 7 + q / 9)))).max() <= 1.7e-8
