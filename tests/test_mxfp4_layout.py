"""quant_mxfp4 and dequant_mxfp4 take their sizes from a tensor and refuse, before
anything is enqueued, what is not laid out as those sizes say (no GPU needed: a
stand-in for the library records the calls)."""
import pytest
import torch

import combine_moe_dispatch_gb300 as moe
from combine_moe_dispatch_gb300 import Status

E, ROWS, COLS = 2, 130, 96


class _Library:
    def __init__(self, monkeypatch, on_gpu=True):
        self.calls = []
        if on_gpu:
            monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t.is_meta else 0)
        monkeypatch.setattr(moe, "load_library", lambda: self)

    def moe_status_string(self, status):
        return b"status"

    def moe_quant_mxfp4(self, *args):
        self.calls.append(args)
        return 0

    moe_dequant_mxfp4 = moe_quant_mxfp4


def _tensors(**other):
    t = dict(wide=torch.zeros((E, ROWS, COLS), dtype=torch.bfloat16),
             q=torch.zeros((E, ROWS, COLS // 2), dtype=torch.uint8),
             scale=torch.zeros((E, 2, 1, 512), dtype=torch.uint8), counts=torch.zeros(E, dtype=torch.int32))
    t.update(other)
    return t


def _both(wide, q, scale, counts):
    return (moe.quant_mxfp4(wide, counts, q, scale, stream=0, check=False),
            moe.dequant_mxfp4(q, scale, counts, wide, stream=0, check=False))


def _refused(**other):
    assert _both(**_tensors(**other)) == (Status.INVALID_ARG, Status.INVALID_ARG), other.keys()


def test_what_fits_is_taken(monkeypatch):
    lib = _Library(monkeypatch)
    ok = (Status.OK, Status.OK)
    for other in ({}, dict(counts=None), dict(scale=torch.zeros(E * 2 * 512, dtype=torch.uint8)),
                  dict(scale=torch.zeros(E * 2 * 512 + 16, dtype=torch.uint8), q=torch.zeros(1 << 14, dtype=torch.int8)),
                  dict(q=torch.zeros((E, ROWS, COLS // 2), dtype=torch.uint8).view(torch.float8_e4m3fn))):
        t = _tensors(**other)
        assert _both(**t) == ok
        quant, back = lib.calls[-2:]
        counts = None if t["counts"] is None else t["counts"].data_ptr()
        assert quant == (E, ROWS, COLS, t["wide"].data_ptr(), counts, 0, t["q"].data_ptr(), t["scale"].data_ptr(), None, 0)
        assert back == (E, ROWS, COLS, t["q"].data_ptr(), t["scale"].data_ptr(), counts, 0, t["wide"].data_ptr(), None, 0)
    # no array at all is the library's to refuse
    assert _both(**_tensors(q=None, scale=None)) == ok and lib.calls[-1][3:5] == (None, None)


def test_other_layouts_are_refused(monkeypatch):
    lib = _Library(monkeypatch)
    bf16 = dict(dtype=torch.bfloat16)
    for wide in (torch.zeros((E, COLS, ROWS), **bf16).transpose(1, 2), torch.zeros((E, 2 * ROWS, COLS), **bf16)[:, ::2],
                 torch.zeros((E, ROWS, 2 * COLS), **bf16)[:, :, :COLS], torch.zeros((1, ROWS, COLS), **bf16).expand(E, -1, -1),
                 torch.zeros((2 * E, ROWS, COLS), **bf16)[::2], torch.zeros((E * ROWS, COLS), **bf16),
                 torch.zeros((1, E, ROWS, COLS), **bf16)):
        _refused(wide=wide)
    for q in (torch.zeros((E, COLS // 2, ROWS), dtype=torch.uint8).transpose(1, 2),
              torch.zeros((E, ROWS, COLS), dtype=torch.uint8)[:, :, ::2]):
        _refused(q=q)
    _refused(scale=torch.zeros((2, E, 1, 512), dtype=torch.uint8).transpose(0, 1))
    _refused(scale=torch.zeros((E, 2, 1, 1024), dtype=torch.uint8)[..., ::2])
    _refused(counts=torch.zeros(2 * E, dtype=torch.int32)[::2])
    assert lib.calls == []
    with pytest.raises(moe.MoEError):
        moe.quant_mxfp4(torch.zeros((E, ROWS, COLS), **bf16)[:, ::2], None, None, None, stream=0)
    with pytest.raises(moe.MoEError):
        moe.dequant_mxfp4(None, None, None, torch.zeros((ROWS, COLS), **bf16), stream=0)


def test_other_types_are_refused(monkeypatch):
    lib = _Library(monkeypatch)
    for dtype in (torch.float16, torch.float32, torch.int16, torch.uint8):
        _refused(wide=torch.zeros((E, ROWS, COLS), dtype=dtype))
    for name in ("q", "scale"):
        _refused(**{name: torch.zeros((E, ROWS, COLS), dtype=torch.int32)})
    for dtype in (torch.int64, torch.int16, torch.float32):
        _refused(counts=torch.zeros(E, dtype=dtype))
    assert lib.calls == []


def test_smaller_arrays_are_refused(monkeypatch):
    lib = _Library(monkeypatch)
    _refused(q=torch.zeros(E * ROWS * COLS // 2 - 1, dtype=torch.uint8))
    _refused(scale=torch.zeros(E * 2 * 512 - 1, dtype=torch.uint8))
    _refused(counts=torch.zeros(E - 1, dtype=torch.int32))
    assert lib.calls == []


def test_host_tensors_are_refused(monkeypatch):
    lib = _Library(monkeypatch, on_gpu=False)
    _refused()
    assert lib.calls == []


def test_two_devices_are_refused(monkeypatch):
    lib = _Library(monkeypatch)
    for name, dims, dtype in (("q", (E, ROWS, COLS // 2), torch.uint8), ("scale", (E, 2, 1, 512), torch.uint8),
                              ("counts", (E,), torch.int32)):
        _refused(**{name: torch.zeros(dims, dtype=dtype, device="meta")})
    assert lib.calls == []
