"""Pins of the 4-bit format's reference (mxfp4_ref), on the CPU: a block worked by
hand, every E2M1 number and border, the places of the scales, and the
measurement's own two forms, written apart from it."""
import importlib.util
import os

import torch

import mxfp4_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _block(values):
    return torch.tensor(list(values) + [0.0] * (32 - len(values)), dtype=torch.float64)[None]


def test_a_block_by_hand():
    # the largest magnitude, 7.5, lies in [4, 8): X = 2^(2 - 2) = 1
    x = [7.5, -7.5, 6.0, 5.0, 5.1, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.26, -0.2, -0.0, 4.9, -1.0]
    q = [6.0, -6.0, 6.0, 4.0, 6.0, 4.0, 2.0, 2.0, 1.0, 1.0, 0.0, 0.5, -0.0, -0.0, 4.0, -1.0]
    code, biased = ref.quantise(_block(x))
    assert biased.tolist() == [[127]]
    got = ref.values(code, biased)[0, :len(x)]
    assert torch.equal(got, torch.tensor(q, dtype=torch.float64))
    assert torch.equal(torch.signbit(got), torch.signbit(torch.tensor(q)))
    # a power of two times the block: the same codes, another scale
    for e in (-140, -100, 37, 100):
        c2, b2 = ref.quantise(_block(x) * 2.0 ** e)
        if e >= -127:
            assert torch.equal(c2, code) and int(b2) == 127 + e
        else:
            assert int(b2) == 0                            # X is never below 2^-127
    # packed: the first element in the low half
    assert ref.pack(code)[0, 0].item() == 7 + 16 * 15
    assert torch.equal(ref.unpack(ref.pack(code)), code)


def test_scales_at_powers_of_two():
    for amax, biased in ((4.0, 127), (7.99, 127), (8.0, 128), (3.99, 126), (2.0 ** -126, 0), (2.0 ** -133, 0),
                         (0.0, 0), (3.3e38, 252), (float("inf"), 255), (float("nan"), 255)):
        assert int(ref.quantise(_block([0.0, amax]))[1]) == biased, amax
    assert bool(ref.values(*ref.quantise(_block([1.0, float("inf")]))).isnan().all())


def test_places():
    # 130 rows of 160: 2 row tiles of 2 block tiles
    at = ref.places(130, 160, False, "cpu")
    assert at[0].tolist() == [0, 1, 2, 3, 512] and at[1, 0] == 16 and at[32, 0] == 4 and at[127, 2] == 31 * 16 + 12 + 2
    assert at[129, 4] == 2 * 512 + 512 + 16
    # gate and up of 65 features: the first 64 of each in one tile, the last ones in the next
    at = ref.places(130, 32, True, "cpu")[:, 0]
    assert at[0] == 0 and at[65] == 8 and at[63] == 31 * 16 + 4 and at[128] == 31 * 16 + 12
    assert at[64] == 512 and at[129] == 512 + 8
    for rows, cols, gate_up in ((130, 160, False), (130, 160, True), (2, 32, True), (256, 128, True)):
        at = ref.places(rows, cols, gate_up, "cpu").reshape(-1)
        assert len(set(at.tolist())) == at.numel()
        assert int(at.max()) < ref.scale_tensor(1, rows, cols, 0, "cpu").numel()


def test_the_measurement_means_the_same():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    g = torch.Generator().manual_seed(1)
    v = torch.randn((2, 130, 96), generator=g) * torch.exp2(torch.randint(-20, 20, (2, 130, 1), generator=g).float())
    v = v.bfloat16().float()
    v[0, 3], v[1, 5, :32] = 0.0, 1e-39
    code, biased = ref.quantise(v)
    q, b = m._quantise(v.view(2, 130, 3, 32))
    assert torch.equal(b.long(), biased) and torch.equal(m._codes(q).view(2, 130, 48), ref.pack(code))
    want = ref.values(code, biased)
    assert torch.equal(m._nearest(v.double().view(-1, 32)).view(v.shape), want)
    for gate_up in (False, True):
        padded = torch.nn.functional.pad(biased, (0, 1))
        scale = ref.place(padded, ref.scale_tensor(2, 130, 96, 0, "cpu"), gate_up)
        assert torch.equal(m._tiled(b.to(torch.uint8), gate_up), scale)
        assert torch.equal(m._untiled(scale, 130, 3, gate_up).long(), biased)
