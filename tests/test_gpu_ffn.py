"""moe_ffn and moe_ffn_backward through the C ABI against the formulas in 64
bits, element by element.

Rows past each expert's count hold NaN in every input, and a sentinel in
every row-wise output that must still be there afterwards.

Tolerances, per element, from the operators' arithmetic: with u = 2^-8 (bf16
has 8 significant bits: round to nearest is off by at most 2^-8, relative)
and sums of K products kept in binary32 (each step at most 2^-23 relative,
whatever its rounding), a result r = sum p_i q_i with an operand p that was
itself rounded to bf16 is off by at most u |r| + (u + K 2^-23) sum |p_i q_i|,
plus what p's own error brings in.  The activation's exponential and quotient are good to 2^-18 for the |gate| < 20
that occur here.  All of it is evaluated in 64 bits from the inputs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
STEP = 2.0 ** -23
ACT = 2.0 ** -18
SENTINEL = -12345.0
D = torch.float64

# E, cap, H, I, counts.  One token of one expert at the smallest sizes; an
# empty expert, one row, a full one; more rows than one tile of 256 columns,
# just over it, and a multiple of 64; sizes that are multiples of 8 alone;
# more experts than a warp has lanes, most of them empty; counts below zero
# and above cap are clamped; few tiles and contractions over 1024 and more,
# which are cut into parts; several tiles of every
# product for each pair of SMs.
SHAPES = [
    (1, 1, 8, 8, [1]),
    (3, 5, 264, 136, [0, 5, 1]),
    (2, 300, 128, 192, [257, 300]),
    (2, 64, 72, 1000, [64, 33]),
    (4, 640, 320, 72, [513, 0, 640, 31]),
    (40, 7, 136, 128, [0] * 31 + [3, 7, 0, 0, 1, 0, 0, 0, 2]),
    (3, 40, 256, 264, [-5, 99, 17]),
    (70, 2, 64, 64, [1, 0, 2] * 23 + [1]),
    (2, 130, 2056, 520, [130, 65]),
    (3, 33, 1040, 2056, [33, 0, 7]),
    (1, 300, 2048, 1096, [290]),
    (8, 64, 1032, 520, [64, 1, 0, 63, 33, 64, 5, 64]),
    (33, 20, 520, 264, [20, 1, 0] * 11),
]
IDS = [f"E{s[0]}-cap{s[1]}-H{s[2]}-I{s[3]}" for s in SHAPES]


def _normal(shape, std, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _case(E, cap, H, I, counts, seed):
    import combine_moe_dispatch_gb300 as moe
    c = [min(max(n, 0), cap) for n in counts]
    x = _normal((E, cap, H), 1.0, seed)
    h = _normal((E, cap, 2 * I), 1.5, seed + 1)
    dy = _normal((E, cap, H), 0.5, seed + 2)
    for e in range(E):
        x[e, c[e]:] = float("nan")
        h[e, c[e]:] = float("nan")
        dy[e, c[e]:] = float("nan")
    wgu = _normal((E, 2 * I, H), H ** -0.5, seed + 3)
    wd = _normal((E, H, I), I ** -0.5, seed + 4)
    shape = moe.make_shape(1, max(1, E * cap), H, E, 1, cap)
    ws = torch.zeros(moe.ffn_workspace_size(shape, I), dtype=torch.uint8, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    return moe, shape, c, x, h, dy, wgu, wd, ws, cnt


def _buf(*dims):
    return torch.full(dims, SENTINEL, dtype=torch.bfloat16, device="cuda")


def _near(got, want, tol, what):
    err = (got.to(D) - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float((err / tol.clamp_min(1e-300)).max()):.3g} tolerances")


def _untouched(t, counts, what):
    for e, n in enumerate(counts):
        assert bool((t[e, n:] == SENTINEL).all()), f"{what}: rows past expert {e}'s count were written"


def _forward64(x, wgu, wd, I):
    """y, h and their tolerances, for one expert's rows."""
    x, wgu, wd = x.to(D), wgu.to(D), wd.to(D)
    H = x.shape[1]
    h = x @ wgu.t()
    dh = H * STEP * (x.abs() @ wgu.abs().t())           # before h's own rounding
    g, u = h[:, :I], h[:, I:]
    sg = torch.sigmoid(g)
    a = g * sg * u
    # |silu'| <= 1.1
    da = ACT * a.abs() + 1.1 * u.abs() * dh[:, :I] + (g * sg).abs() * dh[:, I:] + \
        1.1 * dh[:, :I] * dh[:, I:]
    y = a @ wd.t()
    ab = a.abs() + da
    dy = U * y.abs() + (U + I * STEP) * (1 + U) * (ab @ wd.abs().t()) + (1 + U) * (da @ wd.abs().t())
    return y, dy * (1 + 2 * U), h, (dh + U * (h.abs() + dh)), a, da + U * ab


@pytest.mark.parametrize("E,cap,H,I,counts", SHAPES, ids=IDS)
@pytest.mark.parametrize("keep", [True, False])
def test_ffn(E, cap, H, I, counts, keep):
    moe, shape, c, x, _, _, wgu, wd, ws, cnt = _case(E, cap, H, I, counts, 10)
    h, act, y = _buf(E, cap, 2 * I), _buf(E, cap, I), _buf(E, cap, H)
    moe.ffn(shape, I, x, wgu, wd, cnt, h if keep else None, act, y, ws)
    assert moe.read_status(ws) == moe.Status.OK
    _untouched(act, c, "act")
    _untouched(y, c, "y")
    if keep:
        _untouched(h, c, "h")
    for e, n in enumerate(c):
        if n == 0:
            continue
        y64, ytol, h64, htol, a64, atol = _forward64(x[e, :n], wgu[e], wd[e], I)
        _near(act[e, :n], a64, atol, f"act, expert {e}")
        _near(y[e, :n], y64, ytol, f"y, expert {e}")
        if keep:
            _near(h[e, :n], h64, htol, f"h, expert {e}")


def _backward64(dy, x, h, wgu, wd, I):
    dy, x, h, wgu, wd = (t.to(D) for t in (dy, x, h, wgu, wd))
    n, H = x.shape
    g, u = h[:, :I], h[:, I:]
    sg = torch.sigmoid(g)
    silu, a = g * sg, g * sg * u
    grad = sg * (1.0 + g * (1.0 - sg))
    da = dy @ wd
    eda = H * STEP * (dy.abs() @ wd.abs())
    # 1 + g (1 - s) loses bits where it cancels: its error is relative to its terms
    egrad = ACT * (sg + (silu * (1.0 - sg)).abs())
    dh = torch.cat([da * u * grad, da * silu], 1)
    edh = torch.cat([eda * (u * grad).abs() + (da.abs() + eda) * u.abs() * egrad,
                     eda * silu.abs() + (da.abs() + eda) * silu.abs() * ACT], 1)
    edh = edh + U * (dh.abs() + edh)                    # dh is rounded
    ea = ACT * a.abs()
    ea = ea + U * (a.abs() + ea)

    def product(p, ep, q, K):
        r = p @ q
        e = ep @ q.abs() + K * STEP * ((p.abs() + ep) @ q.abs())
        return r, e + U * (r.abs() + e)

    return (product(dh, edh, wgu, 2 * I), product(dh.t(), edh.t(), x, n),
            tuple(t.t() for t in product(a.t(), ea.t(), dy, n)))


@pytest.mark.parametrize("E,cap,H,I,counts", SHAPES, ids=IDS)
def test_ffn_backward(E, cap, H, I, counts):
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


def test_rows_without_counts():
    """expert_num_tokens = NULL: every expert has cap rows (a dense
    feed-forward); the optional gradients may be left out one by one."""
    E, cap, H, I = 1, 70, 136, 200
    moe, shape, c, x, h, dy, wgu, wd, ws, _ = _case(E, cap, H, I, [cap], 30)
    act, y = _buf(E, cap, I), _buf(E, cap, H)
    moe.ffn(shape, I, x, wgu, wd, None, None, act, y, ws)
    y64, ytol, *_ = _forward64(x[0], wgu[0], wd[0], I)
    _near(y[0], y64, ytol, "y")
    dh, dx = _buf(E, cap, 2 * I), _buf(E, cap, H)
    dwgu, dwd = _buf(E, 2 * I, H), _buf(E, H, I)
    wants = _backward64(dy[0], x[0], h[0], wgu[0], wd[0], I)
    for skip in range(3):
        outs = [dx, dwgu, dwd]
        for t in outs:
            t.fill_(SENTINEL)
        given = [None if i == skip else t for i, t in enumerate(outs)]
        moe.ffn_backward(shape, I, dy, x, h, wgu, wd, None, act, dh, *given, ws)
        for i, t in enumerate(outs):
            if i == skip:
                assert bool((t == SENTINEL).all())
            else:
                _near(t[0], wants[i][0], wants[i][1], f"gradient {i} without {skip}")


def test_gradients_against_differences():
    """The loss sum(y * g) in 64 bits, moved a small step along a random
    direction of x and of each weight: the gradients' inner products with the
    directions agree with the central differences.  The forward pass of the
    differences is the formula's, so its error is the step's (h^2) alone; the
    gradients are off by a few bf16 roundings of a sum with random signs,
    far below the 2 % asked of the inner product's scale."""
    E, cap, H, I, n = 1, 48, 64, 96, 37
    moe, shape, c, x, _, dy, wgu, wd, ws, cnt = _case(E, cap, H, I, [n], 40)
    h, act, y = _buf(E, cap, 2 * I), _buf(E, cap, I), _buf(E, cap, H)
    moe.ffn(shape, I, x, wgu, wd, cnt, h, act, y, ws)
    dh, dx = _buf(E, cap, 2 * I), _buf(E, cap, H)
    dwgu, dwd = _buf(E, 2 * I, H), _buf(E, H, I)
    moe.ffn_backward(shape, I, dy, x, h, wgu, wd, cnt, act, dh, dx, dwgu, dwd, ws)

    def loss(x, wgu, wd):
        g, u = (x @ wgu.t()).split(I, 1)
        return float(((g * torch.sigmoid(g) * u) @ wd.t() * dy[0, :n].to(D)).sum())

    at = [x[0, :n].to(D), wgu[0].to(D), wd[0].to(D)]
    step = 1e-5
    for i, grad in enumerate((dx[0, :n], dwgu[0], dwd[0])):
        v = torch.randn(at[i].shape, dtype=D, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(i))
        up = [t + step * v if j == i else t for j, t in enumerate(at)]
        down = [t - step * v if j == i else t for j, t in enumerate(at)]
        slope = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(float((grad.to(D) * v).sum()) - slope) <= 0.02 * float(grad.to(D).norm()), i


def test_wide_values_and_large_offsets():
    """Gates so large and so small that the exponential overflows or vanishes;
    and a buffer whose last expert lies past 2^31 elements."""
    E, cap, H, I = 9, 8, 64, 64
    moe, shape, c, x, *_ , ws, cnt = _case(E, cap, H, I, [2] * E, 50)
    wgu = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda")
    wgu[:, :I, 0] = 100.0
    wgu[:, I:, 1] = 1.0
    wd = torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    wd[:, torch.arange(H), torch.arange(I)] = 1.0          # y = a
    x[:, :2] = 0
    x[:, 0, 0], x[:, 1, 0] = 50.0, -50.0                   # gate = 5000, -5000
    x[:, :2, 1] = 2.0
    act, y = _buf(E, cap, I), _buf(E, cap, H)
    moe.ffn(shape, I, x, wgu, wd, cnt, None, act, y, ws)
    assert bool((y[:, 0] == 9984.0).all())                 # 10000 rounded to bf16
    assert bool((y[:, 1] == 0).all())
    E, cap, H, I = 5, 65536, 8192, 8                       # E * cap * H = 2.5 * 2^30
    shape = moe.make_shape(1, E * cap, H, E, 1, cap)
    ws = torch.zeros(moe.ffn_workspace_size(shape, I), dtype=torch.uint8, device="cuda")
    x = torch.empty((E, cap, H), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((E, cap, H), dtype=torch.bfloat16, device="cuda")
    y[-1] = SENTINEL
    x[-1, :3] = _normal((3, H), 1.0, 51)
    wgu, wd = _normal((E, 2 * I, H), H ** -0.5, 52), _normal((E, H, I), I ** -0.5, 53)
    act = _buf(E, cap, I)
    cnt = torch.tensor([0, 0, 0, 0, 3], dtype=torch.int32, device="cuda")
    moe.ffn(shape, I, x, wgu, wd, cnt, None, act, y, ws)
    y64, ytol, *_ = _forward64(x[-1, :3], wgu[-1], wd[-1], I)
    _near(y[-1, :3], y64, ytol, "y past 2^31")
    assert bool((y[-1, 3:] == SENTINEL).all())


def test_status_set_writes_nothing_and_stream_order():
    """After a plan error the call writes nothing; on another stream it is
    ordered by that stream alone, also inside a CUDA graph."""
    E, cap, H, I = 4, 20, 128, 128
    moe, shape, c, x, h, dy, wgu, wd, ws, cnt = _case(E, cap, H, I, [3, 20, 0, 7], 60)
    act, y = _buf(E, cap, I), _buf(E, cap, H)
    bad = torch.full((E * cap, 1), E, dtype=torch.int32, device="cuda")
    b = moe.Buffers(shape, expert_x=False, expert_y=False)
    b.workspace = torch.zeros_like(ws)          # one workspace for the plan and the feed-forward
    b.plan(bad)
    assert moe.read_status(b.workspace) == moe.Status.BAD_EXPERT
    moe.ffn(shape, I, x, wgu, wd, cnt, None, act, y, b.workspace)
    dwgu, dwd, dh = _buf(E, 2 * I, H), _buf(E, H, I), _buf(E, cap, 2 * I)
    moe.ffn_backward(shape, I, dy, x, h, wgu, wd, cnt, act, dh, y, dwgu, dwd, b.workspace)
    torch.cuda.synchronize()
    for t in (act, y, dwgu, dwd, dh):
        assert bool((t == SENTINEL).all())
    moe.ffn(shape, I, x, wgu, wd, cnt, None, act, y, ws)
    want = y.clone()
    s = torch.cuda.Stream()
    y2, act2 = _buf(E, cap, H), _buf(E, cap, I)
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.ffn(shape, I, x, wgu, wd, cnt, None, act2, y2, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, want)
    cnt.copy_(torch.tensor([0, 5, 1, 0], dtype=torch.int32))      # counts are read at run time
    y2.fill_(SENTINEL)
    graph.replay()
    torch.cuda.synchronize()
    _untouched(y2, [0, 5, 1, 0], "y")
    assert torch.equal(y2[1, :5], want[1, :5])


def test_one_workspace_for_many_shapes():
    """One workspace serves shapes of every size in turn, with plans of other
    shapes in between: past its header nothing needs to be kept or zero (the
    plan's rows of one shape lie where another's partial sums are)."""
    import combine_moe_dispatch_gb300 as moe
    todo = [SHAPES[i] for i in (9, 5, 12, 10, 9)]
    size = max(moe.ffn_workspace_size(moe.make_shape(1, max(1, E * cap), H, E, 1, cap), I)
               for E, cap, H, I, _ in todo)
    shared = torch.zeros(size, dtype=torch.uint8, device="cuda")
    plan_shape = moe.make_shape(4, 3000, 64, 200, 4, 12000)
    assert moe.workspace_size(plan_shape) <= size
    for k, (E, cap, H, I, counts) in enumerate(todo):
        shared[256:] = 0xFF
        b = moe.Buffers(plan_shape, expert_x=False, expert_y=False)
        b.workspace = shared
        b.plan(torch.randint(0, 200, (12000, 4), dtype=torch.int32, device="cuda"))
        assert moe.read_status(shared) == moe.Status.OK
        _, shape, c, x, h, dy, wgu, wd, _, cnt = _case(E, cap, H, I, counts, 70 + k)
        act, y = _buf(E, cap, I), _buf(E, cap, H)
        moe.ffn(shape, I, x, wgu, wd, cnt, None, act, y, shared)
        dh, dx, dwgu, dwd = _buf(E, cap, 2 * I), _buf(E, cap, H), _buf(E, 2 * I, H), _buf(E, H, I)
        moe.ffn_backward(shape, I, dy, x, h, wgu, wd, cnt, act, dh, dx, dwgu, dwd, shared)
        for e, n in enumerate(c):
            if n == 0:
                continue
            y64, ytol, *_ = _forward64(x[e, :n], wgu[e], wd[e], I)
            _near(y[e, :n], y64, ytol, f"y, shape {k}, expert {e}")
            (rx, ex), (rgu, egu), (rd, ed) = _backward64(dy[e, :n], x[e, :n], h[e, :n], wgu[e], wd[e], I)
            _near(dx[e, :n], rx, ex, f"dx, shape {k}, expert {e}")
            _near(dwgu[e], rgu, egu, f"d_w_gate_up, shape {k}, expert {e}")
            _near(dwd[e], rd, ed, f"d_w_down, shape {k}, expert {e}")
        assert moe.read_status(shared) == moe.Status.OK


@pytest.mark.parametrize("i", [4, 9, 10, 11])
def test_same_bits_every_time(i):
    """Which pair of SMs takes a tile, and which part of a split contraction
    finishes last, differ from run to run; the results do not."""
    E, cap, H, I, counts = SHAPES[i]
    moe, shape, c, x, h, dy, wgu, wd, ws, cnt = _case(E, cap, H, I, counts, 90)
    first = None
    for _ in range(4):
        act, y, dx = _buf(E, cap, I), _buf(E, cap, H), _buf(E, cap, H)
        dh, dwgu, dwd = _buf(E, cap, 2 * I), _buf(E, 2 * I, H), _buf(E, H, I)
        moe.ffn(shape, I, x, wgu, wd, cnt, None, act, y, ws)
        moe.ffn_backward(shape, I, dy, x, h, wgu, wd, cnt, act, dh, dx, dwgu, dwd, ws)
        out = [t.view(torch.int16) for t in (y, act, dh, dx, dwgu, dwd)]
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(out, first))
