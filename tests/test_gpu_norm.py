"""moe_add_rms_norm and its backward pass through the C ABI against the
formulas in 64 bits, element by element.

Tolerances, per element, from the arithmetic: u = 2^-8 is the rounding to bf16
(half a step), relative.  With S = H 2^-23, each step of a binary32 sum of H
terms of one sign being at most 2^-23 relative, mean(s^2) is within S and rstd
within S / 2 + 2^-21 (its square root and reciprocal: 2 units of 2^-23, and the
division and addition before them), relative; y before its rounding adds two
products.  A result below bf16's normal numbers is off by at most half a
subnormal, 2^-134.  Backward, g u is summed with both signs: its mean is within
(2 S + 2^-20) mean |g u|.  d_gain sums N products in binary32."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
TINY = 2.0 ** -134
D = torch.float64
SENTINEL = -12345.0

# N, H: one token; every number of warps a row takes, at its ends and with lanes
# that have nothing; more rows than the grid has places; rows that do not fit
# the registers
SHAPES = [(1, 8), (5, 16), (7, 256), (3, 264), (9, 512), (33, 520), (2, 1024), (17, 1032), (4, 2048),
          (6, 2064), (3, 4096), (5, 4104), (2, 7168), (1, 8192), (3, 8208), (2, 16384), (2, 16400),
          (5, 40000), (6000, 64),
          (2500, 1040), (1300, 7168), (700, 8448), (400, 17408)]
IDS = [f"N{n}-H{h}" for n, h in SHAPES]


def _rand(shape, std, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _near(got, want, tol, what):
    bad = ~((got.to(D) - want).abs() <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float(((got.to(D) - want).abs() / tol).max()):.3g} tolerances")


def _exact(x, r, gain, eps):
    """s, u = s rstd and y, and the relative error of u."""
    s = x.to(D) if r is None else (x.to(D) + r.to(D)).to(torch.bfloat16).to(D)
    H = x.shape[1]
    rstd = (s.square().mean(1, keepdim=True) + eps).rsqrt()
    return s, s * rstd, s * rstd * gain.to(D), rstd, H * 2.0 ** -24 + 2.0 ** -20


def _fp8(moe, y64, off, q, scale, what):
    """E4M3 bytes and scales of y: the scale within y's error, each byte within
    half a step (2^-4 relative, 2^-10 below the normal numbers) of y / scale."""
    N, H = y64.shape
    nb = (H + 127) // 128
    pad = torch.nn.functional.pad(y64, (0, nb * 128 - H)).view(N, nb, 128)
    want = pad.abs().amax(2) / 448.0
    _near(scale, want, want * (off + 2.0 ** -23), what + " scale")
    step = scale.to(D).repeat_interleave(128, 1)[:, :H]
    val = q.view(torch.float8_e4m3fn).to(D) * step
    tol = (2.0 ** -4 + off) * y64.abs() + 2.0 ** -10 * step
    _near(val, y64, tol, what + " bytes")


@pytest.mark.parametrize("N,H", SHAPES, ids=IDS)
@pytest.mark.parametrize("residual", [True, False], ids=["residual", "alone"])
def test_norm(N, H, residual):
    import combine_moe_dispatch_gb300 as moe
    eps = 1e-6
    x, gain = _rand((N, H), 2.0, 1), _rand((H,), 1.0, 2)
    x[N // 2] *= 2.0 ** -60                      # eps decides this row
    if N > 2:
        x[N - 1] = 0.0
    r = _rand((N, H), 1.0, 3) if residual else None
    if residual:
        r[N // 2] *= 2.0 ** -60
    s64, _, y64, _, off = _exact(x, r, gain, eps)
    tol = (U + off) * y64.abs() + TINY
    buf = lambda: torch.full((N, H), SENTINEL, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y, total = buf(), buf() if residual else None
    shape = moe.make_shape(1, N, H, 1, 1, 1)
    moe.add_rms_norm(shape, x, r, gain, eps, total, y)
    _near(y, y64, tol, "y")
    if residual:
        assert torch.equal(total.to(D), s64)
        # the sum not wanted
        y2 = buf()
        moe.add_rms_norm(shape, x, r, gain, eps, None, y2)
        assert torch.equal(y, y2)
    if H % 16:
        return
    nb = (H + 127) // 128
    for payload in (moe.PAYLOAD_FP8_E4M3, moe.PAYLOAD_FP8_E4M3_TSCALE):
        shape8 = moe.make_shape(1, N, H, 1, 1, 1, payload)
        q = torch.full((N, H), 0x7F, dtype=torch.uint8, device="cuda")
        dims = (N, nb) if payload == moe.PAYLOAD_FP8_E4M3 else (nb, N)
        scale = torch.full(dims, SENTINEL, device="cuda")
        y8 = buf()
        moe.add_rms_norm(shape8, x, r, gain, eps, total, y8 if payload == 1 else None, q, scale)
        if payload == 1:
            assert torch.equal(y8, y)
        else:
            scale = scale.t()
        _fp8(moe, y64, off, q, scale, f"payload {payload}")
        if N > 2 and not residual:
            assert bool((q[N - 1] == 0).all()) and bool((scale[N - 1] == 0).all())


@pytest.mark.parametrize("N,H", [(5, 264), (40, 4096), (3, 8208), (3, 16400)])
def test_in_place(N, H):
    """s over x or over the residual, and y over the other one."""
    import combine_moe_dispatch_gb300 as moe
    x, r, gain = _rand((N, H), 1.0, 4), _rand((N, H), 1.0, 5), _rand((H,), 1.0, 6)
    shape = moe.make_shape(1, N, H, 1, 1, 1)
    s, y = torch.empty_like(x), torch.empty_like(x)
    moe.add_rms_norm(shape, x, r, gain, 1e-5, s, y)
    for over in (0, 1):
        a = [x.clone(), r.clone()]
        moe.add_rms_norm(shape, a[0], a[1], gain, 1e-5, a[over], a[1 - over])
        assert torch.equal(a[over], s) and torch.equal(a[1 - over], y)
    a = s.clone()
    moe.add_rms_norm(shape, a, None, gain, 1e-5, None, a)
    assert torch.equal(a, y)


def _backward(N, H, d_sum, seed=7, eps=1e-6):
    import combine_moe_dispatch_gb300 as moe
    s, gain = _rand((N, H), 2.0, seed), _rand((H,), 1.0, seed + 1)
    dy = _rand((N, H), 0.5, seed + 2)
    ds = _rand((N, H), 0.5, seed + 3) if d_sum else None
    shape = moe.make_shape(1, N, H, 1, 1, 1)
    ws = torch.full((moe.norm_workspace_size(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    dx = torch.full((N, H), SENTINEL, dtype=torch.bfloat16, device="cuda")
    dgain = torch.full((H,), SENTINEL, device="cuda")
    call = lambda out=dx, a=dy, b=ds: moe.add_rms_norm_backward(  # noqa: E731
        shape, a, b, s, gain, eps, out, dgain, ws)
    return s, gain, dy, ds, dx, dgain, call


@pytest.mark.parametrize("N,H", SHAPES, ids=IDS)
@pytest.mark.parametrize("d_sum", [True, False], ids=["stream", "alone"])
def test_backward(N, H, d_sum):
    s, gain, dy, ds, dx, dgain, call = _backward(N, H, d_sum)
    call()
    s64, u, _, rstd, off = _exact(s, None, gain, 1e-6)
    g = dy.to(D) * gain.to(D)
    mean = (g * u).mean(1, keepdim=True)
    want = rstd * (g - u * mean)
    dmean = (2 * off + 2.0 ** -20) * (g * u).abs().mean(1, keepdim=True)
    # the terms' own errors before the rounding
    err = rstd * ((2 * off) * (g.abs() + (u * mean).abs()) + u.abs() * dmean)
    if d_sum:
        want = want + ds.to(D)
        err = err + 2.0 ** -23 * want.abs()
    _near(dx, want, U * want.abs() + (1 + U) * err + TINY, "d_x")
    total = (dy.to(D) * u).sum(0)
    _near(dgain, total, (off + N * 2.0 ** -23 + 2.0 ** -22) * (dy.to(D) * u).abs().sum(0) + 1e-30, "d_gain")
    # the same bits again, and in place
    again = dgain.clone()
    for out in (dy.clone(),) + ((ds.clone(),) if d_sum else ()):
        a, b = (out, ds) if out.data_ptr() and torch.equal(out, dy) else (dy, out)
        call(out, a, b)
        assert torch.equal(out, dx) and torch.equal(dgain, again)


def test_backward_against_differences():
    """<dL, direction> against a central difference of the forward formula in 64
    bits, L = <y, c> + <s, c2>."""
    N, H, eps = 6, 392, 1e-6
    s, gain, dy, ds, dx, dgain, call = _backward(N, H, True)
    call()

    def loss(row, w):
        y = row * (row.square().mean(1, keepdim=True) + eps).rsqrt() * w
        return float((y * dy.to(D)).sum() + (row * ds.to(D)).sum())

    g = torch.Generator(device="cuda").manual_seed(99)
    step = 1e-5
    for _ in range(4):
        a = torch.randn(s.shape, dtype=D, device="cuda", generator=g)
        b = torch.randn(gain.shape, dtype=D, device="cuda", generator=g)
        diff = (loss(s.to(D) + step * a, gain.to(D) + step * b) -
                loss(s.to(D) - step * a, gain.to(D) - step * b)) / (2 * step)
        got = float((dx.to(D) * a).sum() + (dgain.to(D) * b).sum())
        # each element of d_x is rounded by at most U of itself (and a hundredth for the rest)
        tol = 1.01 * U * float((dx.to(D) * a).abs().sum()) + 1e-5 * float((dgain.to(D) * b).abs().sum())
        assert abs(got - diff) <= tol


def test_backward_of_an_empty_batch():
    import combine_moe_dispatch_gb300 as moe
    shape = moe.make_shape(2, 0, 264, 1, 1, 1)
    ws = torch.full((moe.norm_workspace_size(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    dgain = torch.full((264,), SENTINEL, device="cuda")
    moe.add_rms_norm_backward(shape, None, None, None, None, 1e-6, None, dgain, ws)
    assert bool((dgain == 0).all())


def test_non_finite_rows_stay_in_their_rows():
    import combine_moe_dispatch_gb300 as moe
    N, H = 20, 1040
    x, gain = _rand((N, H), 1.0, 8), _rand((H,), 1.0, 9)
    shape = moe.make_shape(1, N, H, 1, 1, 1)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    moe.add_rms_norm(shape, x, None, gain, 1e-6, None, y0)
    x[3, 17], x[11, 0], x[12] = float("nan"), float("inf"), 3e38
    moe.add_rms_norm(shape, x, None, gain, 1e-6, None, y1)
    fine = [i for i in range(N) if i not in (3, 11, 12)]
    assert torch.equal(y0[fine], y1[fine])
    assert bool(y1[3].isnan().all())
    assert bool(y1[11, 0].isnan()) and bool((y1[11, 1:] == 0).all())
    assert bool((y1[12] == 0).all())             # squares beyond binary32


def test_captured_and_on_another_stream():
    s, gain, dy, ds, dx, dgain, call = _backward(50, 4096, True)
    import combine_moe_dispatch_gb300 as moe
    shape = moe.make_shape(1, 50, 4096, 1, 1, 1)
    y = torch.empty_like(s)
    call()
    moe.add_rms_norm(shape, s, dy, gain, 1e-6, None, y)
    want = [t.clone() for t in (dx, dgain, y)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            moe.add_rms_norm(shape, s, dy, gain, 1e-6, None, y)
            call()
    for t in (dx, dgain, y):
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (dx, dgain, y)))
