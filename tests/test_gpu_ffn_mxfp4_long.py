"""moe_ffn_mxfp4 where tiles of y have many blocks, on both sides of the length from
which a pair of SMs holds one alone until all of a is written: more tiles of y than
pairs, groups of experts that are empty, and fewer tiles than pairs.  Checked as in
test_gpu_ffn_mxfp4; then the same bits from further calls."""
import pytest

import test_gpu_ffn_mxfp4 as ffn

pytestmark = pytest.mark.gpu

# E, cap, H, I, counts: 27, 28 and 29 blocks of 256
SHAPES = [
    (12, 40, 2048, 6912, [40, 1, 33, 7, 0, 40, 12, 12, 31, 2, 40, 25]),
    (12, 40, 2048, 7168, [3, 40, 0, 40, 17, 40, 1, 1, 40, 32, 33, 40]),
    (20, 9, 1056, 7200, [9, 0, 0] + [0] * 9 + [4, 0, 1, 9, 0, 0, 0, 8]),
    (2, 600, 512, 7200, [600, 257]),
]


@pytest.mark.parametrize("E,cap,H,I,counts", SHAPES, ids=[f"E{s[0]}-cap{s[1]}-H{s[2]}-I{s[3]}" for s in SHAPES])
def test_long_tiles(E, cap, H, I, counts):
    moe, s = ffn._case(E, cap, H, I, counts, 90)
    ffn._run(moe, s)
    assert moe.read_status(s["ws"]) == moe.Status.OK
    ffn._check(s, E, cap, H, I)
    want = ffn._results(s)
    for _ in range(5):
        ffn._clear(s)
        ffn._run(moe, s)
        assert ffn._same(want, ffn._results(s))
    assert moe.read_status(s["ws"]) == moe.Status.OK
