"""Gates so far below zero that their sigmoid is near or below the smallest
normal binary32 number, with values of up that bring the product back.

Tolerance, relative: one rounding to bf16 (2^-8), and the sigmoid's error, with
2^(-g log2 e - 20) for the exponential: half a unit in the last place of an
exponent below 256 (2^-17, times ln 2), of log2 e (133 times 2^-25), 2^-22 for
each of the two approximate instructions, and half of the last place of a
subnormal number above 2^-133 (2^-17): together below 2^-15."""
import pytest
import torch

pytestmark = pytest.mark.gpu

D = torch.float64
GATES = [-60.0, -80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -92.0, -1.0, 0.0, 1.0, 20.0, 88.0, 100.0]
REL = 2.0 ** -8 + 2.0 ** -15


def _near(got, want):
    want = want.expand_as(got)
    assert bool(((got.to(D) - want).abs() <= REL * want.abs()).all()), (got, want)


def _sizes():
    import combine_moe_dispatch_gb300 as moe
    n, H, I = len(GATES), 64, 64
    shape = moe.make_shape(1, n, H, 1, 1, n)
    ws = torch.zeros(moe.ffn_workspace_size(shape, I), dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    return moe, shape, n, H, I, ws, bf


@pytest.mark.parametrize("up", [1.0, 2.0 ** 100])
def test_forward(up):
    moe, shape, n, H, I, ws, bf = _sizes()
    x, wgu = torch.zeros((1, n, H), **bf), torch.zeros((1, 2 * I, H), **bf)
    x[0, :, 0] = torch.tensor(GATES, **bf)
    x[0, :, 1] = up
    wgu[0, :I, 0], wgu[0, I:, 1] = 1.0, 1.0
    act, y = torch.empty((1, n, I), **bf), torch.empty((1, n, H), **bf)
    moe.ffn(shape, I, x, wgu, torch.zeros((1, H, I), **bf), None, None, act, y, ws)
    g = x[0, :, :1].to(D)
    # without up the smallest are below what bf16 holds
    keep = slice(None) if up > 1.0 else (g[:, 0] > -87.0)
    _near(act[0][keep], (g * torch.sigmoid(g) * up)[keep])


def test_backward():
    moe, shape, n, H, I, ws, bf = _sizes()
    up = 2.0 ** 100
    h = torch.empty((1, n, 2 * I), **bf)
    h[0, :, :I] = torch.tensor(GATES, **bf)[:, None]
    h[0, :, I:] = up
    dy, wd = torch.zeros((1, n, H), **bf), torch.zeros((1, H, I), **bf)
    dy[0, :, 0], wd[0, 0] = 1.0, 1.0                       # da = 1
    act, dh = torch.empty((1, n, I), **bf), torch.empty((1, n, 2 * I), **bf)
    dx = torch.empty((1, n, H), **bf)
    moe.ffn_backward(shape, I, dy, torch.zeros((1, n, H), **bf), h, torch.zeros((1, 2 * I, H), **bf), wd,
                     None, act, dh, dx, None, None, ws)
    g = h[0, :, :1].to(D)
    s = torch.sigmoid(g)
    _near(act[0], g * s * up)
    # 1 + g (1 - s) cancels nowhere here (it is 0 at -1.28 alone)
    _near(dh[0, :, :I], up * s * (1.0 + g * torch.sigmoid(-g)))
    # the smallest of dup = SiLU(gate) are below what bf16 holds
    keep = g[:, 0] > -87.0
    _near(dh[0, :, I:][keep], (g * s)[keep])
