"""Limits of the state-space block's entry points that depend on the launch a
call would make.  Runs on the CPU: a call beyond them comes back before
anything is enqueued."""
import os

import pytest

import hyena_long_conv_amd as H
from tests.test_ssm_abi import BIG, P, UNSUP, scan

pytestmark = pytest.mark.skipif(not os.path.exists(H.LIB_PATH), reason="library not built")


def test_scan_backward_counts_the_threads_of_its_workgroups():
    """Beyond 32 states and 16 channels to a group a workgroup has 512 threads: 2^23 of them are 2^32 threads."""
    call = dict(which="hyena_selective_scan_backward", io=1, B=1 << 18, G=16, D=272, N=33, L=129, ws=P[13], wsb=BIG)
    need = H.selective_scan_backward_workspace_bytes(call["B"], call["D"], call["G"], call["N"], call["L"])
    assert 0 < need < BIG
    assert scan(**call) == UNSUP
