"""clip_grad_norm refuses what it cannot walk as one stretch of memory, before
anything is enqueued (no GPU needed: a call that passed the checks would go
on to a launch, which fails here with another status)."""
import ctypes

import pytest

import combine_moe_dispatch_gb300 as moe
from combine_moe_dispatch_gb300 import Status


class _Device:
    """torch.Tensor.is_cuda as if host tensors were on a GPU, and a stand-in
    for the library that records the call's table instead of launching."""

    def __init__(self, monkeypatch):
        import torch
        self.calls = []
        monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
        monkeypatch.setattr(moe, "load_library", lambda: self)

    def moe_status_string(self, status):
        return b"status"

    def moe_clip_grad_norm(self, table, n, max_norm, norm, ws, size, stream):
        self.calls.append((bytes(ctypes.string_at(table, 32 * n)) if n else b"", n))
        return 0


def _call(grads, outs):
    import torch
    ws, norm = torch.zeros(1 << 14, dtype=torch.uint8), torch.zeros(1)
    return moe.clip_grad_norm(grads, outs, 1.0, norm, ws, stream=0, check=False)


def _views(dtype):
    import torch
    buf = torch.zeros((8, 16), dtype=dtype)
    return {"columns": buf[:, :4], "rows apart": buf[::2], "expanded": buf[:, :1].expand(8, 16),
            "a broadcast scalar": torch.zeros((), dtype=dtype).expand(32),
            "a transposed slice": buf[:, :4].t(), "every other": buf.view(-1)[::2]}


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_strided_views_are_refused(monkeypatch, kind):
    import torch
    lib = _Device(monkeypatch)
    good = torch.zeros(8)
    for what, view in _views(getattr(torch, kind)).items():
        flat = torch.zeros(view.numel(), dtype=view.dtype)
        for grads, outs in (([good, view], None), ([flat], [view]), ([view], [flat]),
                            ([view], [view]), ([view, good], [flat, good])):
            got = _call(grads, grads if outs is None else outs)
            assert got == Status.INVALID_ARG, what
    with pytest.raises(moe.MoEError):
        moe.clip_grad_norm([view], [view], 1.0, good, good, stream=0)
    assert lib.calls == []


def test_dense_tensors_are_taken(monkeypatch):
    """Contiguous ones of any shape, and ones that are dense in another order
    where input and output agree; nothing at all."""
    import struct

    import torch
    lib = _Device(monkeypatch)
    a, b = torch.zeros((6, 10)), torch.zeros(60)
    at = torch.zeros((10, 6)).t()
    cube = torch.zeros((3, 4, 5)).permute(2, 0, 1)
    one = torch.zeros((7, 1, 3)).transpose(0, 1)
    for grads, outs in (([a], [b]), ([at], [torch.zeros((10, 6)).t()]), ([cube, a], None),
                        ([one], [torch.zeros((7, 1, 3)).transpose(0, 1)]), ([], []),
                        ([torch.zeros((0, 4))[:, ::2]], None)):
        assert _call(grads, grads if outs is None else outs) == Status.OK
        table, n = lib.calls[-1]
        assert n == len(grads)
        for i, (g, o) in enumerate(zip(grads, grads if outs is None else outs)):
            assert struct.unpack_from("<QQqii", table, 32 * i) == (g.data_ptr(), o.data_ptr(), g.numel(), 1, 0)
    # dense, but not in one order
    assert _call([at], [a]) == Status.INVALID_ARG
    assert _call([at], [b]) == Status.INVALID_ARG
    assert _call([cube], [torch.zeros((5, 3, 4))]) == Status.INVALID_ARG


def test_host_tensors_are_refused():
    import torch
    g = torch.zeros(8)
    assert _call([g], [g]) == Status.INVALID_ARG
    h = [g]
    assert _call(h, h) == Status.INVALID_ARG
