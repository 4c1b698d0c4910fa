"""moe_quant_mxfp4, moe_dequant_mxfp4 and moe_dispatch_mxfp4 through the C ABI.
Everything here is exact: a scale is a power of two read from the largest
magnitude, an element is rounded once, a value of a block is a bf16 number.  So
bytes are compared with the definition's (mxfp4_ref) for equality, and what no
call may touch with the sentinel it held."""
import pytest
import torch

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

FILL = 0xA5


def _rows(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(shape, device="cuda", generator=g)
    t *= torch.exp2(torch.randint(-30, 30, shape[:-1] + (1,), device="cuda", generator=g).float())
    return t.bfloat16()


def _call(src, counts=None, flags=0):
    import combine_moe_dispatch_gb300 as moe
    E, rows, cols = src.shape
    q = torch.full((E, rows, cols // 2), FILL, dtype=torch.uint8, device="cuda")
    scale = ref.scale_tensor(E, rows, cols, FILL)
    assert scale.numel() == moe.mxfp4_scale_bytes(E, rows, cols)
    moe.quant_mxfp4(src, counts, q, scale, flags)
    return q, scale


def _check(src, q, scale, below, flags=0):
    """Every byte of q and scale: the rows below the counts as defined, the
    others as they were."""
    E, rows, cols = src.shape
    code, biased = ref.quantise(src)
    want_q = torch.where(below[..., None], ref.pack(code), torch.full_like(q, FILL))
    assert torch.equal(q, want_q)
    # blocks past the row's end in its last tile are 0
    more = -(cols // 32) % 4
    biased = torch.nn.functional.pad(biased, (0, more))
    biased = torch.where(below[..., None], biased, FILL)
    assert torch.equal(scale, ref.place(biased, ref.scale_tensor(E, rows, cols, FILL), bool(flags)))


def _below(E, rows, counts):
    if counts is None:
        return torch.ones((E, rows), dtype=torch.bool, device="cuda")
    return torch.arange(rows, device="cuda")[None, :] < counts.clamp(0, rows)[:, None]


SHAPES = [(1, 1, 32), (3, 5, 64), (2, 33, 96), (1, 129, 128), (2, 300, 160), (1, 64, 1024), (2, 130, 1056),
          (5, 17, 7168), (40, 3, 2080), (300, 2, 288), (1, 5000, 288)]


@pytest.mark.parametrize("E,rows,cols", SHAPES)
@pytest.mark.parametrize("counted", [False, True])
def test_rows(E, rows, cols, counted):
    import combine_moe_dispatch_gb300 as moe
    src = _rows((E, rows, cols), 1)
    counts = None
    if counted:
        g = torch.Generator(device="cuda").manual_seed(2)
        counts = torch.randint(-2, rows + 3, (E,), device="cuda", generator=g, dtype=torch.int32)
    below = _below(E, rows, counts)
    src[~below] = float("nan")
    q, scale = _call(src, counts)
    _check(src, q, scale, below)
    out = torch.full_like(src, -7.0)
    moe.dequant_mxfp4(q, scale, counts, out)
    code, biased = ref.quantise(src)
    want = torch.where(below[..., None], ref.values(code, biased), -7.0)
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("E,rows,cols", [(1, 2, 32), (2, 64, 96), (1, 128, 128), (3, 130, 288), (2, 1000, 160),
                                         (1, 4096, 1024)])
def test_gate_and_up(E, rows, cols):
    import combine_moe_dispatch_gb300 as moe
    src = _rows((E, rows, cols), 3)
    q, scale = _call(src, flags=moe.MXFP4_GATE_UP)
    _check(src, q, scale, _below(E, rows, None), 1)
    out = torch.empty_like(src)
    moe.dequant_mxfp4(q, scale, None, out, moe.MXFP4_GATE_UP)
    assert torch.equal(out.double(), ref.values(*ref.quantise(src)))


def test_every_bf16_number():
    """Every finite bf16 x in a block whose largest magnitude is x itself, 1.5,
    2.5 and 200 times x: all scales, ties, subnormals and signs."""
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)
    x = x[x.isfinite()]
    src = torch.zeros((1, 4 * len(x), 32), dtype=torch.bfloat16, device="cuda")
    for i, f in enumerate((1.0, 1.5, 2.5, 200.0)):
        part = src[0, i * len(x):(i + 1) * len(x)]
        part[:, 7] = x
        part[:, 20] = (x.float() * f).clamp(-3.3e38, 3.3e38).bfloat16()
        part[:, 31] = -x
    q, scale = _call(src)
    _check(src, q, scale, _below(1, src.shape[1], None))


def test_unaligned_arrays():
    """bf16 arrays at 16 bytes past a boundary of 32, on both sides."""
    import combine_moe_dispatch_gb300 as moe
    for counted in (False, True):
        flat = torch.full((8 + 3 * 40 * 288 + 8,), -7.0, dtype=torch.bfloat16, device="cuda")
        src = flat[8:-8].view(3, 40, 288)
        src.copy_(_rows((3, 40, 288), 12))
        counts = torch.tensor([40, 0, 33], dtype=torch.int32, device="cuda") if counted else None
        below = _below(3, 40, counts)
        q, scale = _call(src, counts)
        _check(src, q, scale, below)
        want = torch.where(below[..., None], ref.values(*ref.quantise(src)), src.double())
        moe.dequant_mxfp4(q, scale, counts, src)
        assert torch.equal(src.double(), want)
        assert bool((flat[:8] == -7.0).all()) and bool((flat[-8:] == -7.0).all())


def test_most_experts():
    """2048 experts with counts, most of them empty; more without."""
    counts = torch.zeros(2048, dtype=torch.int32, device="cuda")
    counts[::77] = 1
    counts[2047] = 3
    src = _rows((2048, 3, 160), 13)
    q, scale = _call(src, counts)
    _check(src, q, scale, _below(2048, 3, counts))
    src = _rows((5000, 1, 64), 14)
    q, scale = _call(src)
    _check(src, q, scale, _below(5000, 1, None))


def test_infinities_and_nan():
    import combine_moe_dispatch_gb300 as moe
    src = _rows((1, 6, 128), 4)
    src[0, 0, 3], src[0, 1, 40], src[0, 2, 64], src[0, 3, 127] = float("inf"), float("-inf"), float("nan"), 3.3e38
    src[0, 4] = 0.0
    src[0, 5] = -0.0
    q, scale = _call(src)
    _check(src, q, scale, _below(1, 6, None))
    out = torch.empty_like(src)
    moe.dequant_mxfp4(q, scale, None, out)
    nan = out.isnan().view(6, 4, 32)
    want = torch.zeros((6, 4), dtype=torch.bool)
    want[0, 0] = want[1, 1] = want[2, 2] = True
    assert torch.equal(nan.all(-1).cpu(), want) and torch.equal(nan.any(-1).cpu(), want)
    assert float(out[0, 3, 127]) == 6.0 * 2.0 ** 125


def test_beyond_32_bits():
    """More than 2^32 bytes of bf16: the last rows, at offsets that 32 bits do
    not hold."""
    import combine_moe_dispatch_gb300 as moe
    E, rows, cols = 3, 40000, 24576
    src = torch.empty((E, rows, cols), dtype=torch.bfloat16, device="cuda")
    src.fill_(1.0)
    src[-1, -3:] = _rows((3, cols), 5)
    q, scale = _call(src)
    tail = src[-1:, -3:].clone()
    code, biased = ref.quantise(tail)
    assert torch.equal(q[-1:, -3:], ref.pack(code))
    at = ref.places(rows, cols, False, "cuda")[-3:]
    assert torch.equal(scale[-1].view(-1)[at].long(), biased[0])
    assert bool((q[0, :1000] == 0x66).all())                   # 1 = 4 * 2^-2
    src.zero_()
    moe.dequant_mxfp4(q, scale, None, src)
    assert torch.equal(src[-1:, -3:].double(), ref.values(code, biased))
    assert bool((src[:-1] == 1.0).all())


def _dispatch(R, T, H, E, K, cap, seed, masked=0.0, idx=None):
    import combine_moe_dispatch_gb300 as moe
    shape = moe.make_shape(R, T, H, E, K, cap)
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = R * T
    if idx is None:
        idx = torch.rand((N, E), device="cuda", generator=g).argsort(1)[:, :K].int()
        idx[torch.rand((N, K), device="cuda", generator=g) < masked] = -1
    x = _rows((N, H), seed + 1)
    b = moe.Buffers(shape, expert_x=False, expert_y=False)
    b.plan_masked(idx.contiguous())
    q = torch.full((E, cap, H // 2), FILL, dtype=torch.uint8, device="cuda")
    scale = ref.scale_tensor(E, cap, H, FILL)
    return moe, shape, x, idx.contiguous(), b, q, scale


def test_dispatch_of_an_unaligned_array():
    moe, shape, x, idx, b, q, scale = _dispatch(1, 64, 288, 8, 2, 64, 15)
    flat = torch.empty(8 + x.numel(), dtype=torch.bfloat16, device="cuda")
    off = flat[8:].view_as(x)
    off.copy_(x)
    moe.dispatch_mxfp4(shape, off, idx, b.slot_of, q, scale, b.workspace)
    q2, scale2 = torch.full_like(q, FILL), torch.full_like(scale, FILL)
    moe.dispatch_mxfp4(shape, x, idx, b.slot_of, q2, scale2, b.workspace)
    assert torch.equal(q, q2) and torch.equal(scale, scale2)


@pytest.mark.parametrize("R,T,H,E,K,cap,masked", [
    (1, 1, 32, 1, 1, 1, 0.0), (1, 64, 256, 8, 2, 64, 0.1), (2, 37, 96, 5, 3, 74, 0.5), (1, 300, 1056, 16, 4, 200, 0.0),
    (8, 128, 7168, 256, 8, 128, 0.0), (1, 5, 160, 40, 32, 5, 0.2), (4, 1000, 64, 3, 1, 4000, 0.0)])
def test_dispatch(R, T, H, E, K, cap, masked):
    moe, shape, x, idx, b, q, scale = _dispatch(R, T, H, E, K, cap, 6, masked)
    moe.dispatch_mxfp4(shape, x, idx, b.slot_of, q, scale, b.workspace)
    assert moe.read_status(b.workspace) == moe.Status.OK
    rows = torch.zeros((E, cap, H), dtype=torch.bfloat16, device="cuda")
    on = b.slot_of >= 0
    token = torch.arange(len(x), device="cuda")[:, None].expand(idx.shape)
    rows[idx[on].long(), b.slot_of[on].long()] = x[token[on]]
    _check(rows, q, scale, _below(E, cap, b.expert_num_tokens))
    # the same as the bf16 dispatch followed by the quantisation of its rows
    ex = torch.empty((E, cap, H), dtype=torch.bfloat16, device="cuda")
    moe.dispatch(shape, x, idx, b.slot_of, ex, None, b.workspace)
    q2, scale2 = torch.full_like(q, FILL), torch.full_like(scale, FILL)
    moe.quant_mxfp4(ex, b.expert_num_tokens, q2, scale2, workspace=b.workspace)
    assert torch.equal(q, q2) and torch.equal(scale, scale2)


def test_dispatch_errors():
    """A failed plan: nothing is written.  Entries out of range: skipped, and
    reported."""
    moe, shape, x, idx, b, q, scale = _dispatch(1, 64, 256, 8, 2, 64, 8)
    bad = idx.clone()
    bad[5, 1] = 8
    b.plan(bad)
    moe.dispatch_mxfp4(shape, x, bad, b.slot_of, q, scale, b.workspace)
    moe.quant_mxfp4(_rows((8, 64, 256), 9), b.expert_num_tokens, q, scale, workspace=b.workspace)
    out = torch.full((8, 64, 256), -7.0, dtype=torch.bfloat16, device="cuda")
    moe.dequant_mxfp4(q, scale, b.expert_num_tokens, out, workspace=b.workspace)
    assert moe.read_status(b.workspace) == moe.Status.BAD_EXPERT
    assert bool((q == FILL).all()) and bool((scale == FILL).all()) and bool((out == -7.0).all())
    for what, value, code in (("idx", 8, moe.Status.BAD_EXPERT), ("idx", -2, moe.Status.BAD_EXPERT),
                              ("slot", 64, moe.Status.CAPACITY), ("slot", -2, moe.Status.CAPACITY)):
        b.plan(idx)
        i, s = idx.clone(), b.slot_of.clone()
        (i if what == "idx" else s)[9, 0] = value
        moe.dispatch_mxfp4(shape, x, i, s, q, scale, b.workspace)
        assert moe.read_status(b.workspace) == code, what


def test_captured_on_another_stream():
    moe, shape, x, idx, b, q, scale = _dispatch(1, 300, 1056, 16, 4, 200, 10)
    out = torch.zeros((16, 200, 1056), dtype=torch.bfloat16, device="cuda")

    def step():
        b.plan(idx)
        moe.dispatch_mxfp4(shape, x, idx, b.slot_of, q, scale, b.workspace)
        moe.dequant_mxfp4(q, scale, b.expert_num_tokens, out, workspace=b.workspace)

    step()
    want = [t.clone() for t in (q, scale, out)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    for t in (q, scale):
        t.fill_(FILL)
    out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, (q, scale, out)))
