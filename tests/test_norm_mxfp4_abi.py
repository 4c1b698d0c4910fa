"""Argument checks of moe_add_rms_norm, its backward pass, MXFP4 quantisation
and moe_dispatch_mxfp4, without a GPU: every call here fails its checks (or has
nothing to do), so that nothing is enqueued and no pointer is followed."""
import ctypes

import pytest

import combine_moe_dispatch_gb300 as moe
from combine_moe_dispatch_gb300 import Shape, Status

A = 0x100000        # an aligned address
B = 0x200000
SHAPE = (1, 16, 256, 4, 2, 16, 0)
FP8 = (1, 16, 256, 4, 2, 16, 1)
EMPTY = (3, 0, 256, 4, 2, 16, 0)


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.load_library()


def _norm(lib, shape=SHAPE, **bad):
    a = dict(x=A, residual=A, gain=A, eps=1e-6, sum=A, y=B, y_q=A, y_scale=A)
    a.update(bad)
    s = Shape(*shape)
    return lib.moe_add_rms_norm(ctypes.byref(s), *a.values(), None)


def test_norm_arguments(lib):
    stop = dict(x=A + 8)                     # what passes the other checks stops here
    for shape in (SHAPE, FP8):
        assert _norm(lib, shape, **stop) == Status.ALIGNMENT
        for name in ("x", "gain"):
            assert _norm(lib, shape, **{name: None}) == Status.INVALID_ARG, name
        for name in ("x", "residual", "gain", "sum", "y"):
            assert _norm(lib, shape, **{name: A + 8}) == Status.ALIGNMENT, name
    # bf16: y is required, the 8-bit arrays are not looked at
    assert _norm(lib, y=None) == Status.INVALID_ARG
    assert _norm(lib, y_q=None, y_scale=A + 2, **stop) == Status.ALIGNMENT
    # fp8: the other way
    assert _norm(lib, FP8, y=None, **stop) == Status.ALIGNMENT
    for name in ("y_q", "y_scale"):
        assert _norm(lib, FP8, **{name: None}) == Status.INVALID_ARG, name
    assert _norm(lib, FP8, y_q=A + 8) == Status.ALIGNMENT
    assert _norm(lib, FP8, y_scale=A + 2) == Status.ALIGNMENT
    # the sum needs a residual, and an array of its own beside y
    assert _norm(lib, residual=None) == Status.INVALID_ARG
    assert _norm(lib, residual=None, sum=None, **stop) == Status.ALIGNMENT
    assert _norm(lib, sum=None, **stop) == Status.ALIGNMENT
    assert _norm(lib, sum=B) == Status.INVALID_ARG
    for eps in (-1e-6, float("nan")):
        assert _norm(lib, eps=eps) == Status.INVALID_ARG
    assert _norm(lib, eps=0.0, **stop) == Status.ALIGNMENT
    assert _norm(lib, (1, 16, 260, 4, 2, 16, 0)) == Status.UNSUPPORTED
    assert _norm(lib, (1, 16, 264, 4, 2, 16, 1)) == Status.UNSUPPORTED       # fp8: H % 16
    assert _norm(lib, EMPTY, x=None, gain=None, y=None) == Status.OK
    assert lib.moe_add_rms_norm(None, *[A] * 3, 1e-6, *[A] * 4, None) == Status.INVALID_ARG


def test_norm_backward_arguments(lib):
    need = moe.norm_workspace_size(Shape(*SHAPE))
    assert need >= 4 * 256

    def call(shape=SHAPE, **bad):
        a = dict(dy=A, dsum=A, sum=A, gain=A, eps=1e-6, dx=A, dgain=A, ws=A, nbytes=need)
        a.update(bad)
        s = Shape(*shape)
        return lib.moe_add_rms_norm_backward(ctypes.byref(s), *a.values(), None)

    for name in ("dy", "sum", "gain", "dx", "dgain"):
        assert call(**{name: None}) == Status.INVALID_ARG, name
    for name in ("dy", "dsum", "sum", "gain", "dx", "ws"):
        assert call(**{name: A + 8}) == Status.ALIGNMENT, name
    assert call(dgain=A + 2) == Status.ALIGNMENT
    assert call(dsum=None, dgain=A + 2) == Status.ALIGNMENT
    assert call(ws=None) == Status.WORKSPACE
    assert call(nbytes=need - 1) == Status.WORKSPACE
    assert call(eps=-1.0) == Status.INVALID_ARG
    assert call(eps=float("nan")) == Status.INVALID_ARG
    for payload in (1, 2):
        assert call(SHAPE[:6] + (payload,)) == Status.UNSUPPORTED
    # an empty batch still has a gradient of the gain: 0
    assert call(EMPTY, dgain=None) == Status.INVALID_ARG
    assert call(EMPTY, dy=None, sum=None, gain=None, dx=None, dgain=A + 2) == Status.ALIGNMENT
    # the workspace is bounded whatever the batch
    assert moe.norm_workspace_size(Shape(8, 1 << 20, 7168, 4, 2, 16, 0)) <= 320 * 4 * 7168
    assert moe.norm_workspace_size(Shape(1, 1, 260, 4, 2, 16, 0)) == 0


def test_scale_bytes(lib):
    assert moe.mxfp4_scale_bytes(1, 1, 32) == 512
    assert moe.mxfp4_scale_bytes(1, 128, 128) == 512
    assert moe.mxfp4_scale_bytes(3, 129, 160) == 3 * 2 * 2 * 512
    assert moe.mxfp4_scale_bytes(256, 4096, 7168) == 256 * 4096 * 7168 // 32
    for bad in ((0, 1, 32), (1, 0, 32), (1, 1, 0), (1, 1, 48), (-1, 1, 32)):
        assert moe.mxfp4_scale_bytes(*bad) == 0


@pytest.mark.parametrize("name", ["moe_quant_mxfp4", "moe_dequant_mxfp4"])
def test_quantisation_arguments(lib, name):
    def call(E=4, rows=16, cols=64, counts=A, flags=0, ws=A, **bad):
        a = dict(src=A, q=A, scale=A)
        a.update(bad)
        f = getattr(lib, name)
        if name == "moe_quant_mxfp4":
            return f(E, rows, cols, a["src"], counts, flags, a["q"], a["scale"], ws, None)
        return f(E, rows, cols, a["q"], a["scale"], counts, flags, a["src"], ws, None)

    stop = dict(src=A + 8)
    assert call(**stop) == Status.ALIGNMENT
    for n in ("src", "q", "scale"):
        assert call(**{n: None}) == Status.INVALID_ARG, n
        assert call(**{n: A + 8}) == Status.ALIGNMENT, n
    assert call(counts=A + 2) == Status.ALIGNMENT
    assert call(ws=A + 8) == Status.ALIGNMENT
    assert call(counts=None, ws=None, **stop) == Status.ALIGNMENT
    for size in ("E", "rows", "cols"):
        assert call(**{size: 0}) == Status.INVALID_ARG
        assert call(**{size: -32}) == Status.INVALID_ARG
    assert call(cols=48) == Status.UNSUPPORTED
    assert call(E=1 << 16, rows=1 << 15, src=None, counts=None) == Status.UNSUPPORTED                  # 2^31 rows
    assert call(E=1 << 16, rows=(1 << 15) - 1, src=None, counts=None) == Status.INVALID_ARG
    assert call(E=1 << 15, rows=1 << 15, cols=1 << 16, src=None, counts=None) == Status.UNSUPPORTED    # 2^46
    assert call(E=1 << 15, rows=1 << 15, cols=(1 << 16) - 32, src=None, counts=None) == Status.INVALID_ARG
    assert call(E=2049, src=None) == Status.UNSUPPORTED                                    # with counts
    assert call(E=2049, counts=None, src=None) == Status.INVALID_ARG
    assert call(E=2048, src=None) == Status.INVALID_ARG
    # the gate and up layout: whole arrays of an even number of rows
    assert call(flags=2) == Status.INVALID_ARG
    assert call(flags=1) == Status.INVALID_ARG                                             # with counts
    assert call(flags=1, counts=None, **stop) == Status.ALIGNMENT
    assert call(flags=1, counts=None, rows=15) == Status.INVALID_ARG


def test_dispatch_mxfp4_arguments(lib):
    def call(shape=SHAPE, **bad):
        a = dict(x=A, idx=A, slot=A, ex=A, scale=A, ws=A)
        a.update(bad)
        s = Shape(*shape)
        return lib.moe_dispatch_mxfp4(ctypes.byref(s), *a.values(), None)

    for n in ("x", "idx", "slot", "ex", "scale"):
        assert call(**{n: None}) == Status.INVALID_ARG, n
    for n, off in (("x", 8), ("ex", 8), ("scale", 8), ("ws", 8), ("idx", 2), ("slot", 2)):
        assert call(**{n: A + off}) == Status.ALIGNMENT, n
    assert call(ws=None) == Status.WORKSPACE
    for payload in (1, 2):
        assert call(SHAPE[:6] + (payload,)) == Status.UNSUPPORTED
    assert call((1, 16, 272, 4, 2, 16, 0)) == Status.UNSUPPORTED             # H % 32
    assert call(EMPTY, x=None, idx=None, slot=None, ex=None, scale=None, ws=None) == Status.OK


I = 128


def _ffn(lib, shape=SHAPE, inter=I, **bad):
    a = dict(x=A, xs=A, wgu=A, wgus=A, wd=A, wds=A, cnt=A, act=A, acts=A, y=A, ws=A, nbytes=1 << 40)
    a.update(bad)
    s = Shape(*shape)
    return lib.moe_ffn_mxfp4(ctypes.byref(s), inter, *a.values(), None)


def test_ffn_mxfp4_arguments(lib):
    required = ["x", "xs", "wgu", "wgus", "wd", "wds", "act", "acts", "y"]
    for name in required:
        assert _ffn(lib, **{name: None}) == Status.INVALID_ARG, name
        assert _ffn(lib, **{name: A + 8}) == Status.ALIGNMENT, name
    assert _ffn(lib, cnt=None, x=A + 8) == Status.ALIGNMENT
    assert _ffn(lib, cnt=A + 2) == Status.ALIGNMENT
    need = moe.ffn_mxfp4_workspace_size(Shape(*SHAPE), I)
    assert _ffn(lib, nbytes=need - 1) == Status.WORKSPACE
    assert _ffn(lib, ws=None) == Status.WORKSPACE
    assert _ffn(lib, ws=A + 8) == Status.ALIGNMENT
    assert _ffn(lib, nbytes=need, x=A + 8) == Status.ALIGNMENT
    assert _ffn(lib, inter=0) == Status.INVALID_ARG
    assert _ffn(lib, inter=-32) == Status.INVALID_ARG
    assert _ffn(lib, inter=144) == Status.UNSUPPORTED                        # not a multiple of 32
    assert _ffn(lib, shape=(1, 16, 272, 4, 2, 16, 0)) == Status.UNSUPPORTED  # H % 32
    for payload in (1, 2):
        assert _ffn(lib, shape=SHAPE[:6] + (payload,)) == Status.UNSUPPORTED


def test_ffn_mxfp4_size_limits(lib):
    """Each limit just passed, and just kept (the call then fails at the next
    check, a null pointer)."""
    null = dict(x=None)
    big = (1, 4, 256, 1024, 2, 1 << 20, 0)                 # E * cap = 2^30
    assert _ffn(lib, big, 1 << 15, **null) == Status.UNSUPPORTED             # rows * 2I = 2^46
    assert _ffn(lib, big, (1 << 15) - 32, **null) == Status.INVALID_ARG
    assert _ffn(lib, (1, 4, 1 << 16, 1024, 2, 1 << 20, 0), 32, **null) == Status.UNSUPPORTED
    assert _ffn(lib, (1, 4, (1 << 16) - 32, 1024, 2, 1 << 20, 0), 32, **null) == Status.INVALID_ARG
    one = (1, 4, 1 << 20, 1, 1, 1, 0)                      # 4 I H = 2^40
    assert _ffn(lib, one, 1 << 18, **null) == Status.UNSUPPORTED
    assert _ffn(lib, one, (1 << 18) - 32, **null) == Status.INVALID_ARG
    thin = (1, 4, 32, 1, 1, 1, 0)
    assert _ffn(lib, thin, 1 << 29, **null) == Status.UNSUPPORTED
    assert _ffn(lib, (1, 4, 1 << 30, 1, 1, 1, 0), 32, **null) == Status.UNSUPPORTED


def test_ffn_mxfp4_workspace_size(lib):
    s = Shape(*SHAPE)
    assert moe.ffn_mxfp4_workspace_size(s, I) >= moe.workspace_size(s)
    assert moe.ffn_mxfp4_workspace_size(s, 0) == 0
    assert moe.ffn_mxfp4_workspace_size(Shape(1, 16, 260, 4, 2, 16, 0), I) == 0
    big = Shape(8, 512, 7168, 256, 8, 8192, 0)             # bounded: sums of 128 tiles of 256 x 256 floats
    assert moe.ffn_mxfp4_workspace_size(big, 2048) <= moe.workspace_size(big) + (128 << 18)
