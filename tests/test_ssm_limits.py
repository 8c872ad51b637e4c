"""Limits of the state-space block's entry points that depend on the launch a
call would make.  Runs on the CPU: a call beyond them comes back before
anything is enqueued."""
import os

import pytest

import hyena_long_conv_amd as H
from tests.test_ssm_abi import ALIAS, BIG, P, SHAPE, UNSUP, scan

pytestmark = pytest.mark.skipif(not os.path.exists(H.LIB_PATH), reason="library not built")


def test_scan_backward_counts_the_threads_of_its_workgroups():
    """Beyond 32 states and 16 channels to a group a workgroup has 512 threads: 2^23 of them are 2^32 threads."""
    call = dict(which="hyena_selective_scan_backward", io=1, B=1 << 18, G=16, D=272, N=33, L=129, ws=P[13], wsb=BIG)
    need = H.selective_scan_backward_workspace_bytes(call["B"], call["D"], call["G"], call["N"], call["L"])
    assert 0 < need < BIG
    assert scan(**call) == UNSUP


def test_product_counts_its_rows_together():
    """Row-major, only B * L is limited; channel-major, the sequences' limits hold."""
    f = lambda B, L, cm, out=P[4]: H.lib().hyena_scaled_matmul(  # noqa: E731
        P[0], P[1], P[2], P[3], None, out, B, L, 32, 16, cm, 1, None)
    assert f((1 << 20) + 1, 8, 0, P[0]) == ALIAS and f(1, (1 << 22) + 1, 0, P[0]) == ALIAS   # past the sizes
    assert f((1 << 20) + 1, 8, 1) == SHAPE and f(1, (1 << 22) + 1, 1) == SHAPE
    assert f(1, (1 << 31) + 1, 0) == SHAPE and f((1 << 31) + 1, 1, 0) == SHAPE and f(1 << 16, (1 << 15) + 1, 0) == SHAPE
    assert f(1 << 62, 1 << 62, 0) == SHAPE
