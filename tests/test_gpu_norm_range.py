"""moe_add_rms_norm and its backward pass over the range of bf16: rows whose
squares binary32 does not hold, with eps so small (0 among them) that the rows
alone decide, against the formulas in 64 bits; and where the range ends.

Tolerances as in test_gpu_norm: multiplying a row by a power of two adds no
rounding, so that sums, root and products err as for rows of ordinary size."""
import pytest
import torch

import test_gpu_norm as base

pytestmark = pytest.mark.gpu

D = torch.float64
U, TINY = base.U, base.TINY
# every number of warps a row takes, lanes that have nothing, rows that do not fit the registers
WIDTHS = [16, 256, 512, 1024, 1040, 2048, 2064, 4096, 7168, 8192, 8208, 16384, 16400]
EPS = [0.0, 2.0 ** -149, 3e-42, 1e-38, 1e-30, 1.1e-28]
# magnitudes: squares that vanish, that lose bits and that are ordinary; eps of the list beside them
EXPONENTS = [-20, -45, -50, -60, -64, -70, -74, -75, -90, -110, -120, -127, -131, 0, 40]


def _rows(H, seed):
    """Normal rows of every magnitude; one of a single smallest number, one
    with a large element among small ones, one of subnormal numbers."""
    N = len(EXPONENTS) + 3
    x = base._rand((N, H), 1.0, seed, torch.float32)
    x[:len(EXPONENTS)] *= torch.exp2(torch.tensor(EXPONENTS, device="cuda", dtype=torch.float32))[:, None]
    x[-3] = 0.0
    x[-3, H // 3] = 2.0 ** -133
    x[-2] *= 2.0 ** -80
    x[-2, H - 2] = 2.0 ** -40
    x[-1] *= 2.0 ** -128
    return x.bfloat16()


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("eps", EPS)
def test_small_rows(H, eps):
    import combine_moe_dispatch_gb300 as moe
    x, gain = _rows(H, 1), base._rand((H,), 1.0, 2)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    for residual in (False, True):
        r = (x.float() * 0.5).bfloat16() if residual else None
        s64, _, y64, _, off = base._exact(x, r, gain, eps)
        N = x.shape[0]
        tol = (U + off) * y64.abs() + TINY
        y, total = torch.empty_like(x), torch.empty_like(x) if residual else None
        moe.add_rms_norm(moe.make_shape(1, N, H, 1, 1, 1), x, r, gain, eps, total, y)
        base._near(y, y64, tol, "y")
        if residual:
            assert torch.equal(total.to(D), s64)
        q = torch.empty((N, H), dtype=torch.uint8, device="cuda")
        scale = torch.empty((N, (H + 127) // 128), device="cuda")
        y8 = torch.empty_like(y)
        moe.add_rms_norm(moe.make_shape(1, N, H, 1, 1, 1, 1), x, r, gain, eps, None, y8, q, scale)
        assert torch.equal(y8, y)
        on = y64.abs().amax(1) > 2.0 ** -100     # (below, the scales themselves are subnormal)
        base._fp8(moe, y64[on], off, q[on], scale[on], "E4M3")


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("d_sum", [True, False], ids=["stream", "alone"])
def test_backward_of_small_rows(H, eps, d_sum):
    """d_x of rows of 2^-133 is 2^133 times d_y: gradients that keep it finite."""
    import combine_moe_dispatch_gb300 as moe
    s, gain = _rows(H, 3), base._rand((H,), 1.0, 4)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    N = s.shape[0]
    dy = base._rand((N, H), 2.0 ** -24, 5)
    ds = base._rand((N, H), 1.0, 6) if d_sum else None
    shape = moe.make_shape(1, N, H, 1, 1, 1)
    ws = torch.full((moe.norm_workspace_size(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dgain = torch.empty_like(s), torch.empty(H, device="cuda")
    moe.add_rms_norm_backward(shape, dy, ds, s, gain, eps, dx, dgain, ws)
    _, u, _, rstd, off = base._exact(s, None, gain, eps)
    g = dy.to(D) * gain.to(D)
    mean = (g * u).mean(1, keepdim=True)
    want = rstd * (g - u * mean)
    dmean = (2 * off + 2.0 ** -20) * (g * u).abs().mean(1, keepdim=True)
    err = rstd * ((2 * off) * (g.abs() + (u * mean).abs()) + u.abs() * dmean)
    if d_sum:
        want = want + ds.to(D)
        err = err + 2.0 ** -23 * want.abs()
    assert float(want.abs().max()) < 2.0 ** 127
    base._near(dx, want, U * want.abs() + (1 + U) * err + TINY, "d_x")
    base._near(dgain, (dy.to(D) * u).sum(0),
               (off + N * 2.0 ** -23 + 2.0 ** -22) * (dy.to(D) * u).abs().sum(0) + 1e-30, "d_gain")


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_where_the_range_ends(eps):
    """A sum of squares below 2^128 is binary32's; from there on the row is 0.
    A row of zeros is 0 / sqrt(eps)."""
    import combine_moe_dispatch_gb300 as moe
    for H in (512, 2048, 7168, 16400):
        x, gain = torch.zeros((3, H), dtype=torch.bfloat16, device="cuda"), base._rand((H,), 1.0, 7)
        edge = 2.0 ** 64 / H ** 0.5
        x[0], x[1] = 0.9 * edge, 1.1 * edge
        y = torch.empty_like(x)
        moe.add_rms_norm(moe.make_shape(1, 3, H, 1, 1, 1), x, None, gain, eps, None, y)
        _, _, y64, _, off = base._exact(x[:1], None, gain, eps)
        base._near(y[:1], y64, (U + off) * y64.abs() + TINY, "y")
        assert bool((y[1] == 0.0).all())
        assert bool(y[2].isnan().all()) if eps == 0.0 else bool((y[2] == 0.0).all())
