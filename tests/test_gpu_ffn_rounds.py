"""moe_ffn and moe_ffn_backward where the row products' tiles fill the SM pairs more
than once, and where the tiles of the last round are cut into parts of their
contraction: a (the activation), y and da (the backward pass's first product), each cut
alone and after whole rounds, with token tiles of several widths.

Which of it happens follows from the tile counts, restated here: 256 tokens by 128
(gate and up) or 256 features, and the kernel's price of a cut.  Tolerances are those
of the element-wise tests of the same calls."""
import pytest
import torch

from test_gpu_ffn import D, _backward64, _buf, _case, _forward64, _near, _untouched

pytestmark = pytest.mark.gpu

# E, cap, H, I, counts, and how a, y and da are cut on 76 pairs: 'Z' all tiles, 'W'
# after whole rounds, '-' not, lower case 'w' not cut but more than one round
SHAPES = [
    (2, 40, 2280, 1632, [33, 20], "ZZZ"),
    (1, 700, 3024, 2912, [600], "-ZZ"),                    # three token tiles of 224 columns
    (1, 700, 2776, 3312, [600], "WZ-"),
    (11, 20, 1784, 1752, [20, 1, 7, 20, 20, 3, 20, 20, 9, 20, 2], "WWW"),
    (4, 300, 3272, 3312, [300, 257, 0, 290], "WWW"),       # uneven tiles of one expert
    (7, 130, 4568, 1392, [130, 65, 3, 20, 31, 32, 1], "Ww-"),   # contractions of 72 blocks, 8 parts
    (8, 64, 4104, 4104, [40, 3, 33, 64, 1, 17, 40, 9], "Www"),  # three rounds of long tiles
    (6, 300, 1032, 2056, [300, 257, 0, 299, 40, 300], "w-w"),
    (9, 33, 1480, 3120, [33, 12, 5, 0, 33, 30, 1, 2, 8], "w-w"),
]
IDS = [f"E{s[0]}-cap{s[1]}-H{s[2]}-I{s[3]}-{s[5]}" for s in SHAPES]


def _cut(counts, features, per_tile, K, pairs):
    """'Z', 'W', 'w' or '-' for a product of `features` outputs over K."""
    tiles = sum(-(-c // 256) for c in counts) * -(-features // per_tile)
    nk, left = -(-K // 64), tiles % pairs
    cols = min(256, -(-max(counts) // 32) * 32)
    price = {}
    for s in range(1, 9):
        if s == 1 or (s * left <= 128 and 4 * s <= nk):
            price[s] = (2 if s * left > pairs else 1) * (-(-nk // s) + 6)
            price[s] += 14 + s * -(-cols // 64) if s > 1 else 0
    parts = min(price, key=lambda s: (price[s], s)) if left and K >= 1024 else 1
    if parts == 1:
        return "w" if tiles > pairs else "-"
    return "W" if tiles > pairs else "Z"


def _check_cuts(H, I, counts, cuts):
    pairs = min(128, torch.cuda.get_device_properties(0).multi_processor_count // 2)
    got = _cut(counts, I, 128, H, pairs) + _cut(counts, H, 256, I, pairs) + _cut(counts, I, 256, H, pairs)
    if pairs == 76:
        assert got == cuts, f"the shape does not do what it is listed for: {got}"


@pytest.mark.parametrize("E,cap,H,I,counts,cuts", SHAPES, ids=IDS)
def test_forward(E, cap, H, I, counts, cuts):
    _check_cuts(H, I, counts, cuts)
    moe, shape, c, x, _, _, wgu, wd, ws, cnt = _case(E, cap, H, I, counts, 10)
    h, act, y = _buf(E, cap, 2 * I), _buf(E, cap, I), _buf(E, cap, H)
    moe.ffn(shape, I, x, wgu, wd, cnt, h, act, y, ws)
    assert moe.read_status(ws) == moe.Status.OK
    for t, what in ((act, "act"), (y, "y"), (h, "h")):
        _untouched(t, c, what)
    for e, n in enumerate(c):
        if n == 0:
            continue
        y64, ytol, h64, htol, a64, atol = _forward64(x[e, :n], wgu[e], wd[e], I)
        _near(act[e, :n], a64, atol, f"act, expert {e}")
        _near(h[e, :n], h64, htol, f"h, expert {e}")
        _near(y[e, :n], y64, ytol, f"y, expert {e}")


@pytest.mark.parametrize("E,cap,H,I,counts,cuts", SHAPES, ids=IDS)
def test_backward(E, cap, H, I, counts, cuts):
    moe, shape, c, x, h, dy, wgu, wd, ws, cnt = _case(E, cap, H, I, counts, 20)
    act, dh, dx = _buf(E, cap, I), _buf(E, cap, 2 * I), _buf(E, cap, H)
    dwgu, dwd = _buf(E, 2 * I, H), _buf(E, H, I)
    moe.ffn_backward(shape, I, dy, x, h, wgu, wd, cnt, act, dh, dx, dwgu, dwd, ws)
    assert moe.read_status(ws) == moe.Status.OK
    for t, what in ((act, "act"), (dh, "dh"), (dx, "dx")):
        _untouched(t, c, what)
    for e, n in enumerate(c):
        if n == 0:
            assert bool((dwgu[e] == 0).all()) and bool((dwd[e] == 0).all()), f"expert {e} has no rows"
            continue
        (rx, ex), (rgu, egu), (rd, ed) = _backward64(dy[e, :n], x[e, :n], h[e, :n], wgu[e], wd[e], I)
        _near(dx[e, :n], rx, ex, f"dx, expert {e}")
        _near(dwgu[e], rgu, egu, f"d_w_gate_up, expert {e}")
        _near(dwd[e], rd, ed, f"d_w_down, expert {e}")


@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 5])
def test_same_bits_every_time(i):
    """The parts of a cut tile finish in any order and are joined in one; the
    workspace's counters serve one call after another."""
    E, cap, H, I, counts, _ = SHAPES[i]
    moe, shape, c, x, h, dy, wgu, wd, ws, cnt = _case(E, cap, H, I, counts, 90)
    runs = []
    for _ in range(6):
        act, y, dx = _buf(E, cap, I), _buf(E, cap, H), _buf(E, cap, H)
        dh, dwgu, dwd = _buf(E, cap, 2 * I), _buf(E, 2 * I, H), _buf(E, H, I)
        moe.ffn(shape, I, x, wgu, wd, cnt, None, act, y, ws)
        first = act.clone()
        moe.ffn_backward(shape, I, dy, x, h, wgu, wd, cnt, act, dh, dx, dwgu, dwd, ws)
        runs.append([t.view(torch.int16) for t in (first, y, act, dh, dx, dwgu, dwd)])
    assert moe.read_status(ws) == moe.Status.OK
    for run in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(run, runs[0]))
