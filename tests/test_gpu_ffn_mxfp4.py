"""moe_ffn_mxfp4 through the C ABI against the formulas in 64 bits, element by
element, in two steps: the 4-bit activations against the exact SiLU(gate) * up,
then y against the product of the activations that the call itself wrote.

Rows past each expert's count hold NaN scales and any bytes, and every output a
sentinel that must still be there afterwards.

Tolerances, per element.  A sum of H products kept in binary32 (each step at
most 2^-23 relative, whatever its rounding) is off by at most H 2^-23 times the
sum of magnitudes; the activation's exponential and quotient are good to 2^-18.
With v = a / X the exact quotient and d the distance of v to the nearest E2M1
number, an element quantised from a value that is off by e (in units of X) is
within d + 2 e of v.  The scale is X of the block's largest magnitude: the exact
one's, or its neighbour where e takes the magnitude past a power of two.  y is
rounded to bf16 once: 2^-8 of itself, and the sum's error."""
import pytest
import torch

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
STEP = 2.0 ** -23
ACT = 2.0 ** -18
FILL = 0xA5
SENTINEL = -12345.0
D = torch.float64

# E, cap, H, I, counts.  One token of one expert at the smallest sizes; an empty
# expert, one row, a full one; more rows than one tile of 256 columns, just over
# it; sizes that are odd multiples of a block of 32; more experts than a warp has
# lanes, most of them empty; counts below zero and above cap are clamped; few
# tiles and contractions over 4096 and more, which are cut into parts; several
# tiles for each pair of SMs whose accumulators share columns, with wide tiles
# before narrow ones and after them.
SHAPES = [
    (1, 1, 32, 32, [1]),
    (3, 5, 288, 160, [0, 5, 1]),
    (1, 32, 256, 128, [32]),
    (1, 200, 128, 64, [200]),
    (2, 300, 128, 192, [257, 300]),
    (2, 64, 96, 992, [64, 33]),
    (4, 640, 320, 96, [513, 0, 640, 31]),
    (40, 7, 160, 128, [0] * 31 + [3, 7, 0, 0, 1, 0, 0, 0, 2]),
    (3, 40, 256, 288, [-5, 99, 17]),
    (70, 2, 64, 64, [1, 0, 2] * 23 + [1]),
    (2, 130, 2080, 544, [130, 65]),
    (3, 33, 1056, 2080, [33, 0, 7]),
    (1, 300, 4096, 1120, [290]),
    (1, 20, 5152, 4128, [20]),
    (33, 20, 544, 288, [20, 1, 0] * 11),
    (3, 1100, 512, 4096, [1024, 777, 1100]),
    (5, 260, 288, 4128, [256, 260, 225, 224, 30]),
]
IDS = [f"E{s[0]}-cap{s[1]}-H{s[2]}-I{s[3]}" for s in SHAPES]


def _quantised(E, rows, cols, std, seed, gate_up=False):
    """Random MXFP4 rows: bytes, scale tiles and what they stand for."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn((E, rows, cols), device="cuda", generator=g) * std
    code, biased = ref.quantise(v)
    scale = ref.place(torch.nn.functional.pad(biased, (0, -(cols // 32) % 4)),
                      ref.scale_tensor(E, rows, cols, 0xFF), gate_up)
    return ref.pack(code), scale, ref.values(code, biased)


def _case(E, cap, H, I, counts, seed):
    import combine_moe_dispatch_gb300 as moe
    c = [min(max(n, 0), cap) for n in counts]
    xq, xs, x = _quantised(E, cap, H, 1.0, seed)
    at = ref.places(cap, H, False, "cuda")
    for e in range(E):                       # rows that do not exist: NaN
        xs[e].view(-1)[at[c[e]:].reshape(-1)] = 255
    wgu = _quantised(E, 2 * I, H, H ** -0.5, seed + 1, True)
    wd = _quantised(E, H, I, I ** -0.5, seed + 2)
    shape = moe.make_shape(1, max(1, E * cap), H, E, 1, cap)
    s = dict(shape=shape, c=c, I=I, xq=xq, xs=xs, x=x, wgu=wgu, wd=wd,
             cnt=torch.tensor(counts, dtype=torch.int32, device="cuda"),
             ws=torch.zeros(moe.ffn_mxfp4_workspace_size(shape, I), dtype=torch.uint8, device="cuda"),
             act=torch.full((E, cap, I // 2), FILL, dtype=torch.uint8, device="cuda"),
             act_scale=ref.scale_tensor(E, cap, I, FILL),
             y=torch.full((E, cap, H), SENTINEL, dtype=torch.bfloat16, device="cuda"))
    return moe, s


def _run(moe, s, cnt="cnt"):
    moe.ffn_mxfp4(s["shape"], s["I"], s["xq"], s["xs"], s["wgu"][0], s["wgu"][1], s["wd"][0], s["wd"][1],
                  s[cnt] if cnt else None, s["act"], s["act_scale"], s["y"], s["ws"])


def _check(s, E, cap, H, I):
    grid = torch.tensor(ref.GRID, dtype=D, device="cuda")
    blocks = -(-I // 128) * 4
    at = ref.places(cap, blocks * 32, False, "cuda")
    scales = s["act_scale"].view(E, -1)[:, at.reshape(-1)].view(E, cap, blocks).long()
    for e, n in enumerate(s["c"]):
        assert bool((s["act"][e, n:] == FILL).all()), f"act: rows past expert {e}'s count were written"
        assert bool((scales[e, n:] == FILL).all()), f"scales: rows past expert {e}'s count were written"
        assert bool((s["y"][e, n:] == SENTINEL).all()), f"y: rows past expert {e}'s count were written"
        if n == 0:
            continue
        assert bool((scales[e, :n, I // 32:] == 0).all()), "blocks past the row's end"
        x, w = s["x"][e, :n], s["wgu"][2][e]
        h = x @ w.t()
        dh = H * STEP * (x.abs() @ w.abs().t())
        g, u = h[:, :I], h[:, I:]
        silu = g * torch.sigmoid(g)
        a = silu * u
        da = ACT * a.abs() + 1.1 * u.abs() * dh[:, :I] + silu.abs() * dh[:, I:] + 1.1 * dh[:, :I] * dh[:, I:]
        biased = scales[e, :n, :I // 32]
        amax = a.abs().view(n, -1, 32)
        err = da.view(n, -1, 32).amax(-1)
        low = (torch.frexp((amax.amax(-1) - err).clamp(min=2.0 ** -130)).exponent - 3 + 127).clamp(min=0)
        high = (torch.frexp(amax.amax(-1) + err).exponent - 3 + 127).clamp(min=0)
        assert bool(((biased >= low) & (biased <= high)).all()), "activation scales"
        power = ref.power(biased - 127).repeat_interleave(32, -1)
        a4 = ref.values(ref.unpack(s["act"][e, :n]), biased)
        v = (a / power).abs()
        dist = (v[..., None] - grid).abs().amin(-1)
        # a largest magnitude next to a power of two may have had the smaller scale
        tol = dist + 2 * da / power
        bad = ~((a4 - a).abs() / power <= tol * (1 + 1e-12))
        assert not bool(bad.any()), f"expert {e}: {int(bad.sum())} of {bad.numel()} activations off"
        wd = s["wd"][2][e]
        y = a4 @ wd.t()
        tol = U * y.abs() + (1 + U) * I * STEP * (a4.abs() @ wd.abs().t()) + 1e-30
        off = (s["y"][e, :n].to(D) - y).abs()
        assert bool((off <= tol).all()), (f"expert {e}: y off, {int((off > tol).sum())} of {off.numel()}, worst "
                                          f"{float((off / tol).max()):.3g} tolerances")


@pytest.mark.parametrize("E,cap,H,I,counts", SHAPES, ids=IDS)
def test_ffn(E, cap, H, I, counts):
    moe, s = _case(E, cap, H, I, counts, 20)
    _run(moe, s)
    assert moe.read_status(s["ws"]) == moe.Status.OK
    _check(s, E, cap, H, I)
    want = [s[k].clone() for k in ("act", "act_scale", "y")]
    for _ in range(3):                       # the same bits again, on the same workspace
        for k, f in (("act", FILL), ("act_scale", FILL), ("y", SENTINEL)):
            s[k].fill_(f)
        _run(moe, s)
        assert all(torch.equal(w, s[k]) for w, k in zip(want, ("act", "act_scale", "y")))


def _clear(s):
    for k, f in (("act", FILL), ("act_scale", FILL), ("y", SENTINEL)):
        s[k].fill_(f)


def _untouched(s):
    return bool((s["act"] == FILL).all()) and bool((s["act_scale"] == FILL).all()) and \
        bool((s["y"] == SENTINEL).all())


def _results(s):
    return [s[k].clone() for k in ("act", "act_scale", "y")]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_without_counts():
    moe, s = _case(3, 33, 256, 160, [33] * 3, 30)
    _run(moe, s)
    want = _results(s)
    _clear(s)
    _run(moe, s, cnt=None)
    assert _same(want, _results(s))


def test_rows_keep_to_themselves():
    """NaN and infinity in one block of two tokens: their rows alone."""
    moe, s = _case(2, 70, 256, 160, [70, 9], 31)
    _run(moe, s)
    want = _results(s)
    at = ref.places(70, 256, False, "cuda")
    s["xs"][0].view(-1)[at[5, 3]] = 255
    s["xs"][0].view(-1)[at[69, 0]] = 254                   # times 6: beyond binary32
    s["xq"][0, 69, :16] = 0x77
    _run(moe, s)
    fine = [i for i in range(70) if i not in (5, 69)]
    assert torch.equal(s["y"][0, fine], want[2][0, fine]) and torch.equal(s["y"][1], want[2][1])
    assert bool(s["y"][0, 5].isnan().all())
    assert not bool(s["y"][0, 69].isfinite().any())


def test_beyond_32_bits():
    """Weights of more than 2^32 bytes; the last expert alone has rows."""
    import combine_moe_dispatch_gb300 as moe
    E, cap, H, I = 44, 40, 7168, 14336
    _, one = _case(1, cap, H, I, [37], 32)
    s = dict(one, c=[0] * (E - 1) + [37], shape=moe.make_shape(1, E * cap, H, E, 1, cap))
    s["cnt"] = torch.tensor(s["c"], dtype=torch.int32, device="cuda")

    def widen(t, fill):
        w = torch.full((E, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")
        w[-1] = t[0]
        return w

    s["xq"], s["xs"] = widen(one["xq"], 0), widen(one["xs"], 255)
    s["wgu"] = (widen(one["wgu"][0], 0), widen(one["wgu"][1], 255))
    s["wd"] = (widen(one["wd"][0], 0), widen(one["wd"][1], 255))
    assert s["wgu"][0].numel() > 2 ** 32
    for k in ("act", "act_scale", "y"):
        s[k] = widen(one[k], FILL if k != "y" else SENTINEL)
    s["ws"] = torch.zeros(moe.ffn_mxfp4_workspace_size(s["shape"], I), dtype=torch.uint8, device="cuda")
    _run(moe, s)
    assert moe.read_status(s["ws"]) == moe.Status.OK
    assert bool((s["y"][:-1] == SENTINEL).all()) and bool((s["act"][:-1] == FILL).all())
    last = dict(one, c=[37], act=s["act"][-1:], act_scale=s["act_scale"][-1:], y=s["y"][-1:])
    _check(last, 1, cap, H, I)


# WsHeader: the status is word 4, flags word 5, the counters start at word 10
FLAGS, NEXT_UNIT = 5, 10
BROKEN = -2 ** 31


def _planned(seed=33):
    """The case of 12 tokens over 2 experts, 2 x 2 tiles of a and 2 of y."""
    moe, s = _case(2, 8, 128, 256, [6, 6], seed)
    s["shape"] = moe.make_shape(1, 12, 128, 2, 1, 8)
    b = moe.Buffers(s["shape"], expert_x=False, expert_y=False)
    b.workspace = s["ws"] = torch.zeros(moe.ffn_mxfp4_workspace_size(s["shape"], 256), dtype=torch.uint8,
                                        device="cuda")
    idx = torch.tensor([[i % 2] for i in range(12)], dtype=torch.int32, device="cuda")

    def step(bad=False):
        b.plan(torch.full_like(idx, 2) if bad else idx)
        _run(moe, s)
        return moe.read_status(s["ws"])

    return moe, s, b, idx, step


def test_failed_plan():
    moe, s, _, _, step = _planned()
    assert step(bad=True) == moe.Status.BAD_EXPERT and _untouched(s)
    assert step() == moe.Status.OK
    _check(s, 2, 8, 128, 256)


def test_wait_that_runs_out():
    """The launch's unit counter is set past the tiles of a, so that nobody
    computes them and the tiles of y wait, 20 ms at most, for a count that
    nothing raises: the kernel returns, reports TIMEOUT and writes nothing, and so
    do later calls until the workspace is initialised."""
    moe, s, b, idx, step = _planned()
    assert step() == moe.Status.OK
    want = _results(s)
    moe.workspace_set_debug(s["ws"], 0, 20_000_000)
    _clear(s)
    b.plan(idx)
    s["ws"].view(torch.int32)[NEXT_UNIT] = 4
    _run(moe, s)
    assert moe.read_status(s["ws"]) == moe.Status.TIMEOUT and _untouched(s)
    moe.workspace_set_debug(s["ws"], 0, 0)
    for _ in range(2):
        assert step() == moe.Status.TIMEOUT and _untouched(s)
    moe.workspace_init(s["ws"])
    assert step() == moe.Status.OK and _same(want, _results(s))


def test_refused_with_the_mark_of_another_call():
    """A wait of moe_ffn that ran out stops this call too."""
    moe, s, _, _, step = _planned()
    _clear(s)
    s["ws"].view(torch.int32)[FLAGS] = BROKEN
    assert step() == moe.Status.TIMEOUT and _untouched(s)


@pytest.mark.parametrize("graph", [False, True])
def test_back_to_back_with_the_bf16_calls(graph):
    """Calls of different shapes, and moe_ffn between them, on one workspace:
    each gives what it gives alone."""
    import combine_moe_dispatch_gb300 as moe
    cases = [_case(*c, 40 + 3 * i)[1] for i, c in enumerate(
        [(1, 1, 32, 32, [1]), (3, 40, 288, 160, [40, 0, 7]), (1, 300, 160, 96, [290]), (2, 4, 64, 64, [0, 0]),
         (1, 20, 5152, 4128, [20]), (90, 2, 64, 96, [1, 2, 0] * 30)])]
    E, cap, H, I = 3, 40, 264, 136
    x = torch.randn((E, cap, H), device="cuda").bfloat16()
    wgu, wd = torch.randn((E, 2 * I, H), device="cuda").bfloat16(), torch.randn((E, H, I), device="cuda").bfloat16()
    act, y = torch.zeros((E, cap, I), device="cuda").bfloat16(), torch.zeros((E, cap, H), device="cuda").bfloat16()
    shape = moe.make_shape(1, E * cap, H, E, 1, cap)
    size = max([moe.ffn_workspace_size(shape, I)] + [s["ws"].numel() for s in cases])
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def bf16():
        moe.ffn(shape, I, x, wgu, wd, None, None, act, y, ws)

    want = []
    for s in cases:
        _run(moe, s)
        want.append(_results(s))
        _clear(s)
        s["ws"] = ws
    bf16()
    y_want = y.clone()

    def run():
        for s in cases:
            _run(moe, s)
            bf16()
            _run(moe, s)

    if graph:
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            run()
        run_it = g.replay
    else:
        run_it = run
    for _ in range(10):
        for s in cases:
            _clear(s)
        y.zero_()
        run_it()
        torch.cuda.synchronize()
        assert moe.read_status(ws) == moe.Status.OK
        assert all(_same(w, _results(s)) for w, s in zip(want, cases)) and torch.equal(y, y_want)


def test_two_streams_at_once():
    """Two calls with workspaces of their own that share the GPU."""
    import combine_moe_dispatch_gb300 as moe
    cases = [_case(3, 600, 512, 1056, [600, 33, 500], 70)[1], _case(40, 30, 1056, 544, [30, 0, 7, 16] * 10, 73)[1]]
    want = []
    for s in cases:
        _run(moe, s)
        want.append(_results(s))
        _clear(s)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                _run(moe, s)
    torch.cuda.synchronize()
    for s, w in zip(cases, want):
        assert moe.read_status(s["ws"]) == moe.Status.OK and _same(w, _results(s))
