"""The longest rows that moe_add_rms_norm and its backward pass take, without a
GPU: every call here fails its checks, the last of them a null pointer's.  From
2^31 - 127 elements on, the kernels' count of 128-element blocks passed 32
bits; rows end well before."""
import ctypes

import pytest

import combine_moe_dispatch_gb300 as moe
from combine_moe_dispatch_gb300 import Shape, Status

A, B = 0x100000, 0x200000
LIMIT = 1 << 30
KEPT = [LIMIT - 16, 1 << 29, 16]
PASSED = [LIMIT, LIMIT + 16, (1 << 31) - 128, (1 << 31) - 112, (1 << 31) - 32, (1 << 31) - 16]


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.load_library()


@pytest.mark.parametrize("payload", [0, 1, 2])
def test_norm(lib, payload):
    for H, want in [(h, Status.INVALID_ARG) for h in KEPT] + [(h, Status.UNSUPPORTED) for h in PASSED]:
        s = Shape(1, 2, H, 1, 1, 1, payload)
        assert lib.moe_add_rms_norm(ctypes.byref(s), None, A, A, 1e-6, A, B, A, A, None) == want, H


def test_norm_backward(lib):
    for H, want in [(h, Status.INVALID_ARG) for h in KEPT] + [(h, Status.UNSUPPORTED) for h in PASSED]:
        s = Shape(1, 2, H, 1, 1, 1, 0)
        assert lib.moe_add_rms_norm_backward(ctypes.byref(s), None, A, A, A, 1e-6, A, A, A, 1 << 62,
                                             None) == want, H
        assert moe.norm_workspace_size(s) == (2 * 4 * H if want == Status.INVALID_ARG else 0)
