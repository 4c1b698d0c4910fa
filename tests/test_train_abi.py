"""Argument checks of moe_ffn, moe_ffn_backward, moe_combine_backward and
moe_clip_grad_norm, without a GPU: every call here fails its checks (or has
nothing to do), so that nothing is enqueued and no pointer is followed."""
import array
import ctypes
import struct

import pytest

import combine_moe_dispatch_gb300 as moe
from combine_moe_dispatch_gb300 import Shape, Status

A = 0x100000        # an aligned address


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.load_library()


SHAPE = (1, 16, 256, 4, 2, 16, 0)
I = 128


def _ffn(lib, shape=SHAPE, inter=I, **bad):
    s = Shape(*shape)
    a = dict(x=A, wgu=A, wd=A, cnt=A, h=A, act=A, y=A, ws=A, nbytes=1 << 40)
    a.update(bad)
    return lib.moe_ffn(ctypes.byref(s), inter, a["x"], a["wgu"], a["wd"], a["cnt"], a["h"],
                 a["act"], a["y"], a["ws"], a["nbytes"], None)


def _backward(lib, shape=SHAPE, inter=I, **bad):
    s = Shape(*shape)
    a = dict(dy=A, x=A, h=A, wgu=A, wd=A, cnt=A, act=A, dh=A, dx=A, dwgu=A, dwd=A, ws=A, nbytes=1 << 40)
    a.update(bad)
    return lib.moe_ffn_backward(ctypes.byref(s), inter, *[a[k] for k in a if k not in ("ws", "nbytes")],
                 a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("call,required,optional", [
    (_ffn, ["x", "wgu", "wd", "act", "y"], ["cnt", "h"]),
    (_backward, ["dy", "x", "h", "wgu", "wd", "act", "dh"], ["cnt", "dx", "dwgu", "dwd"])])
def test_ffn_arguments(lib, call, required, optional):
    for name in required:
        assert call(lib, **{name: None}) == Status.INVALID_ARG, name
        assert call(lib, **{name: A + 8}) == Status.ALIGNMENT, name
    for name in optional:
        # absent is allowed: the call goes on to the next check
        assert call(lib, **{name: None, required[0]: A + 8}) == Status.ALIGNMENT, name
        off = 2 if name == "cnt" else 8
        assert call(lib, **{name: A + off}) == Status.ALIGNMENT, name
    need = moe.ffn_workspace_size(Shape(*SHAPE), I)
    assert call(lib, nbytes=need - 1) == Status.WORKSPACE
    assert call(lib, ws=None) == Status.WORKSPACE
    assert call(lib, ws=A + 8) == Status.ALIGNMENT
    assert call(lib, nbytes=need, **{required[0]: A + 8}) == Status.ALIGNMENT
    assert call(lib, inter=0) == Status.INVALID_ARG
    assert call(lib, inter=-8) == Status.INVALID_ARG
    assert call(lib, inter=132) == Status.UNSUPPORTED                       # not a multiple of 8
    for payload in (1, 2):
        assert call(lib, shape=(1, 16, 256, 4, 2, 16, payload)) == Status.UNSUPPORTED
    assert call(lib, shape=(1, 16, 260, 4, 2, 16, 0)) == Status.UNSUPPORTED  # H % 8
    assert call(lib, shape=(1, 16, 256, 4, 2, 0, 0)) == Status.INVALID_ARG


@pytest.mark.parametrize("call", [_ffn, _backward])
def test_ffn_size_limits(lib, call):
    """Each limit just passed, and just kept (the call then fails at the next
    check, a null pointer)."""
    big = (1, 4, 256, 1024, 2, 1 << 20, 0)                 # E * cap = 2^30
    null = dict(x=None)
    assert call(lib, shape=big, inter=1 << 15, **null) == Status.UNSUPPORTED      # rows * 2I = 2^46
    assert call(lib, shape=big, inter=(1 << 15) - 8, **null) == Status.INVALID_ARG
    wide = (1, 4, 1 << 16, 1024, 2, 1 << 20, 0)            # rows * H = 2^46
    assert call(lib, shape=wide, inter=8, **null) == Status.UNSUPPORTED
    assert call(lib, shape=(1, 4, (1 << 16) - 8, 1024, 2, 1 << 20, 0), inter=8, **null) == Status.INVALID_ARG
    one = (1, 4, 1 << 20, 1, 1, 1, 0)                      # 4 I H = 2^40
    assert call(lib, shape=one, inter=1 << 18, **null) == Status.UNSUPPORTED
    assert call(lib, shape=one, inter=(1 << 18) - 8, **null) == Status.INVALID_ARG
    assert call(lib, shape=(1, 4, 2147483640, 1, 1, 1, 0), inter=2147483640, **null) == Status.UNSUPPORTED
    thin = (1, 4, 8, 1, 1, 1, 0)
    assert call(lib, shape=thin, inter=1 << 29, **null) == Status.UNSUPPORTED
    assert call(lib, shape=thin, inter=(1 << 29) - 8, **null) == Status.INVALID_ARG
    assert call(lib, shape=(1, 4, 1 << 30, 1, 1, 1, 0), inter=8, **null) == Status.UNSUPPORTED
    assert call(lib, shape=(1, 4, (1 << 30) - 8, 1, 1, 1, 0), inter=8, **null) == Status.INVALID_ARG


def test_ffn_workspace_size(lib):
    s = Shape(*SHAPE)
    assert moe.ffn_workspace_size(s, I) >= moe.workspace_size(s)
    assert moe.ffn_workspace_size(s, 0) == 0
    assert moe.ffn_workspace_size(Shape(1, 16, 260, 4, 2, 16, 0), I) == 0
    # bounded whatever the shape: sums of 128 tiles of 256 x 256 floats, four tensor
    # maps per expert, counters
    big = Shape(8, 512, 7168, 256, 8, 8192, 0)
    assert moe.ffn_workspace_size(big, 2048) <= moe.workspace_size(big) + (128 << 18) + 4 * 128 * 256 + 4096


def test_combine_backward_arguments(lib):
    names = ["dy", "ey", "idx", "slot", "w", "dey", "dw", "dl"]
    wide = {"dy": 16, "ey": 16, "dey": 16}

    def call(shape=SHAPE, **bad):
        s = Shape(*shape)
        a = dict.fromkeys(names, A)
        a["ws"] = A
        a.update(bad)
        return lib.moe_combine_backward(ctypes.byref(s), *[a[n] for n in names], a["ws"], None)

    for n in names:
        if n != "dl":
            assert call(**{n: None}) == Status.INVALID_ARG, n
        assert call(**{n: A + (8 if n in wide else 2)}) == Status.ALIGNMENT, n
    assert call(dl=None, dy=A + 8) == Status.ALIGNMENT
    assert call(ws=None) == Status.WORKSPACE
    assert call(ws=A + 8) == Status.ALIGNMENT
    assert call(shape=(1, 16, 256, 4, 33, 16, 0)) == Status.UNSUPPORTED
    assert call(shape=(1, 0, 256, 4, 2, 16, 0), **dict.fromkeys(names)) == Status.OK   # empty batch


def _table(rows):
    t = array.array("q", [v for r in rows for v in r])
    return t, t.buffer_info()[0]


def test_grad_tensor_layout():
    """The binding fills moe_grad_tensor as four 64-bit words: two pointers,
    the count, and the type with a zero word above it."""
    assert struct.calcsize("<QQqii") == 32
    t, _ = _table([(A, A, 5, 1)])
    assert struct.unpack("<QQqii", t.tobytes()) == (A, A, 5, 1, 0)


def test_clip_arguments(lib):
    need = moe.clip_workspace_size()

    def call(rows, num=None, max_norm=1.0, norm=A, ws=A, nbytes=need):
        t, at = _table(rows)
        return lib.moe_clip_grad_norm(at if rows else None, len(rows) if num is None else num,
                                      max_norm, norm, ws, nbytes, None)

    good = (A, A, 8, 0)
    stop = dict(ws=A + 8)                    # what passes the other checks stops here
    assert call([good], **stop) == Status.ALIGNMENT
    assert call([], **stop) == Status.ALIGNMENT
    assert call([good], num=-1) == Status.INVALID_ARG
    assert call([], num=1) == Status.INVALID_ARG
    assert call([good], norm=None) == Status.INVALID_ARG
    assert call([good], max_norm=-1.0) == Status.INVALID_ARG
    assert call([good], max_norm=float("nan")) == Status.INVALID_ARG
    assert call([good, (A, A, -1, 0)]) == Status.INVALID_ARG
    assert call([good, (A, A, 8, 2)]) == Status.INVALID_ARG
    assert call([good, (0, A, 8, 0)]) == Status.INVALID_ARG
    assert call([good, (A, 0, 8, 0)]) == Status.INVALID_ARG
    assert call([good, (0, 0, 0, 0)], **stop) == Status.ALIGNMENT          # an empty tensor is fine
    assert call([(A, A, 1 << 46, 0)]) == Status.UNSUPPORTED
    assert call([(A + 1, A, 8, 0)]) == Status.ALIGNMENT
    assert call([(A + 2, A + 6, 8, 0)], **stop) == Status.ALIGNMENT        # bf16: any even address
    assert call([(A + 2, A, 8, 1)]) == Status.ALIGNMENT
    assert call([good], norm=A + 2) == Status.ALIGNMENT
    assert call([good], ws=None) == Status.WORKSPACE
    assert call([good], nbytes=need - 1) == Status.WORKSPACE


def test_clip_binding_refuses_mixed_lists(lib):
    import torch
    a = torch.zeros(8)
    ws, norm = torch.zeros(moe.clip_workspace_size(), dtype=torch.uint8), torch.zeros(1)
    for grads, outs in (([a], []), ([a], [a.bfloat16()]), ([a], [a[:4]]),
                        ([a.half()], [a.half()])):
        assert moe.clip_grad_norm(grads, outs, 1.0, norm, ws, stream=0, check=False) == Status.INVALID_ARG
        with pytest.raises(moe.MoEError):
            moe.clip_grad_norm(grads, outs, 1.0, norm, ws, stream=0)
