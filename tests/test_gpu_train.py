"""moe_combine_backward and moe_clip_grad_norm through the C ABI against the
formulas in 64 bits.

Tolerances.  Combine: w * dy is one binary32 product (2^-24) and one rounding
to bf16 (2^-8): (2^-8 + 2^-23) |w dy|.  A dot product over H elements in
binary32 is off by at most H 2^-24 of the sum of its terms' magnitudes (its
products are exact).  d_logits: the dot products' errors, weighted, and K + 4
binary32 operations on them.  Norm: binary32 over at most 128 squares
(2^-24 each), half of it through the root, and one rounding: 2^-16 relative.
Clipped values: the norm's error, three binary32 operations and the
rounding to the tensor's type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D = torch.float64
SENTINEL = -12345.0
U24 = 2.0 ** -24
U8 = 2.0 ** -8


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, std, seed, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=_gen(seed))


def _near(got, want, tol, what):
    err = (got.to(D) - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float((err / tol.clamp_min(1e-300)).max()):.3g} tolerances")


# R, T, H, E, K: one token; one warp's row and less; rows of one block; K that
# is not a power of two, more than one group of 8, and the largest; a row that
# ends inside a block's step
SHAPES = [(1, 1, 8, 1, 1), (1, 3, 256, 8, 2), (2, 70, 512, 16, 3), (1, 40, 520, 16, 4),
          (2, 33, 1032, 64, 6), (1, 300, 7168, 32, 8), (1, 21, 2056, 40, 11), (1, 9, 72, 64, 32),
          (1, 5, 4096, 33, 32)]


@pytest.mark.parametrize("R,T,H,E,K", SHAPES)
@pytest.mark.parametrize("masked", [0.0, 0.4])
@pytest.mark.parametrize("logits", [True, False])
def test_combine_backward(R, T, H, E, K, masked, logits):
    import combine_moe_dispatch_gb300 as moe
    N = R * T
    shape = moe.make_shape(R, T, H, E, K, N)
    idx = torch.rand((N, E), device="cuda", generator=_gen(1)).argsort(1)[:, :K].int().contiguous()
    if masked:
        idx[torch.rand((N, K), device="cuda", generator=_gen(2)) < masked] = -1
        idx[N // 2] = -1                                   # a token with nothing routed
    b = moe.Buffers(shape, expert_x=False, expert_y=False)
    b.plan_masked(idx)
    w = torch.softmax(_normal((N, K), 1.0, 3, torch.float32), 1)
    if masked:
        w[idx < 0] = float("nan")                          # weights of such entries are not used
    dy, ey = _normal((N, H), 1.0, 4), _normal((E, N, H), 1.0, 5)
    for e, n in enumerate(b.expert_num_tokens.tolist()):
        ey[e, n:] = float("nan")
    dey = torch.full((E, N, H), SENTINEL, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((N, K), SENTINEL, dtype=torch.float32, device="cuda")
    dl = torch.full((N, E), SENTINEL, dtype=torch.float32, device="cuda")
    moe.combine_backward(shape, dy, ey, idx, b.slot_of, w, dey, dw, dl if logits else None, b.workspace)
    assert moe.read_status(b.workspace) == moe.Status.OK
    routed = b.slot_of >= 0
    e = torch.where(routed, idx, 0).long()
    s = torch.where(routed, b.slot_of, 0).long()
    rows = torch.where(routed[:, :, None], ey[e, s].to(D), 0.0)
    w64 = torch.where(routed, w.to(D), 0.0)
    want = w64[:, :, None] * dy.to(D)[:, None, :]
    _near(dey[e, s][routed], want[routed], (U8 + 2 * U24) * want[routed].abs() + 1e-40, "d_expert_y")
    for i, n in enumerate(b.expert_num_tokens.tolist()):
        assert bool((dey[i, n:] == SENTINEL).all()), "rows past the count were written"
    dw64 = (rows * dy.to(D)[:, None, :]).sum(2)
    mag = (rows * dy.to(D)[:, None, :]).abs().sum(2)
    tol = H * U24 * mag
    _near(dw, dw64, tol, "d_weights")
    if not logits:
        assert bool((dl == SENTINEL).all())
        return
    mean = (w64 * dw64).sum(1, keepdim=True)
    dl64 = torch.zeros((N, E), dtype=D, device="cuda").scatter_add_(1, e, w64 * (dw64 - mean))
    spread = (w64 * (dw64.abs() + tol)).sum(1, keepdim=True)
    t = w64 * (tol + (w64 * tol).sum(1, keepdim=True) + (K + 4) * U24 * (dw64.abs() + tol + spread))
    tol_l = torch.zeros((N, E), dtype=D, device="cuda").scatter_add_(1, e, t)
    _near(dl, dl64, tol_l, "d_logits")


def test_combine_backward_twice_chosen_and_out_of_range():
    """An expert chosen twice by a token gets the sum in d_logits; entries out
    of range are skipped and reported; after an error nothing is written."""
    import combine_moe_dispatch_gb300 as moe
    N, H, E, K = 6, 64, 4, 3
    shape = moe.make_shape(1, N, H, E, K, 2 * N)
    idx = torch.tensor([[1, 1, 3]] * N, dtype=torch.int32, device="cuda")
    b = moe.Buffers(shape, expert_x=False, expert_y=False)
    b.plan(idx)
    w = torch.softmax(_normal((N, K), 1.0, 6, torch.float32), 1)
    dy, ey = _normal((N, H), 1.0, 7), _normal((E, 2 * N, H), 1.0, 8)
    dey = torch.full((E, 2 * N, H), SENTINEL, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((N, K), SENTINEL, dtype=torch.float32, device="cuda")
    dl = torch.full((N, E), SENTINEL, dtype=torch.float32, device="cuda")
    moe.combine_backward(shape, dy, ey, idx, b.slot_of, w, dey, dw, dl, b.workspace)
    rows = ey[idx.long(), b.slot_of.long()].to(D)
    dw64 = (rows * dy.to(D)[:, None, :]).sum(2)
    own = w.to(D) * (dw64 - (w.to(D) * dw64).sum(1, keepdim=True))
    dl64 = torch.zeros((N, E), dtype=D, device="cuda").scatter_add_(1, idx.long(), own)
    mag = (rows * dy.to(D)[:, None, :]).abs().sum(2).max()
    _near(dl, dl64, torch.full_like(dl64, 4 * H * U24 * float(mag)), "d_logits")
    bad = idx.clone()
    bad[2, 1] = E
    dey.fill_(SENTINEL)
    moe.combine_backward(shape, dy, ey, bad, b.slot_of, w, dey, dw, dl, b.workspace)
    assert moe.read_status(b.workspace) == moe.Status.BAD_EXPERT
    dey.fill_(SENTINEL)
    dw.fill_(SENTINEL)
    moe.combine_backward(shape, dy, ey, idx, b.slot_of, w, dey, dw, dl, b.workspace)
    torch.cuda.synchronize()
    assert bool((dey == SENTINEL).all()) and bool((dw == SENTINEL).all())


def _clip(grads, outs, max_norm, ws=None):
    import combine_moe_dispatch_gb300 as moe
    norm = torch.full((1,), SENTINEL, dtype=torch.float32, device="cuda")
    if ws is None:
        ws = torch.zeros(moe.clip_workspace_size(), dtype=torch.uint8, device="cuda")
    moe.clip_grad_norm(grads, outs, max_norm, norm, ws)
    return norm


def _clip_check(grads, max_norm, inplace, ws=None):
    outs = grads if inplace else [torch.full_like(g, SENTINEL) for g in grads]
    before = [g.clone() for g in grads]
    norm = _clip(grads, outs, max_norm, ws)
    want = sum(float(g.to(D).square().sum()) for g in before) ** 0.5
    assert abs(float(norm) - want) <= 2.0 ** -16 * want
    coef = min(1.0, max_norm / (want + 1e-6))
    for o, g in zip(outs, before):
        u = U24 if g.dtype == torch.float32 else U8
        _near(o, g.to(D) * coef, (u + 2.0 ** -15) * (g.to(D) * coef).abs() + 1e-40, "clipped")
    if not inplace:
        for a, g in zip(before, grads):
            assert torch.equal(a, g)
    return norm


SIZES = [[1], [7, 1, 9], [4096], [16384, 16385, 3], [100003, 5, 262144, 31], [0, 12, 0], [8192] * 40]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(s[:3]) for s in SIZES])
@pytest.mark.parametrize("kind", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("max_norm,inplace", [(0.5, False), (0.5, True), (1e6, False), (1e6, True), (0.0, False)])
def test_clip(sizes, kind, max_norm, inplace):
    types = {"bf16": [torch.bfloat16], "fp32": [torch.float32], "mixed": [torch.bfloat16, torch.float32]}[kind]
    grads = [_normal((n,), 1.0, i, types[i % len(types)]) for i, n in enumerate(sizes)]
    _clip_check(grads, max_norm, inplace)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_clip_any_alignment(dtype):
    """Views at every offset of a 16-byte group, in and out offset alike and
    differently; what lies beside a view is not written."""
    n, pad = 40000, 16
    step = 16 // torch.empty((), dtype=dtype).element_size()
    flat = _normal((step * (n + 2 * pad),), 1.0, 9, dtype)
    for shift in (0, 1, 3):
        grads, outs, at = [], [], []
        out = torch.full_like(flat, SENTINEL)
        for i in range(step):
            a = i * (n + 2 * pad) + pad + i
            grads.append(flat[a:a + n - 2 * step])
            outs.append(out[a + shift:a + shift + n - 2 * step])
            at.append((a + shift, a + shift + n - 2 * step))
        norm = _clip(grads, outs, 3.0)
        want = sum(float(g.to(D).square().sum()) for g in grads) ** 0.5
        assert abs(float(norm) - want) <= 2.0 ** -16 * want
        u = U24 if dtype == torch.float32 else U8
        for o, g in zip(outs, grads):
            w = g.to(D) * (3.0 / (want + 1e-6))
            _near(o, w, (u + 2.0 ** -15) * w.abs() + 1e-40, "clipped")
        free = torch.ones(flat.shape, dtype=torch.bool, device="cuda")
        for a, z in at:
            free[a:z] = False
        assert bool((out[free] == SENTINEL).all())


def test_clip_many_tensors_repeats_and_special_values():
    """More tensors than one launch takes; the same bits every time, from a
    workspace that is used again; no tensor at all; NaN and infinity."""
    import combine_moe_dispatch_gb300 as moe
    ws = torch.zeros(moe.clip_workspace_size(), dtype=torch.uint8, device="cuda")
    grads = [_normal((1 + 37 * (i % 50),), 1.0, i, torch.bfloat16 if i % 3 else torch.float32)
             for i in range(1300)]
    first = _clip_check(grads, 1.0, False, ws)
    for _ in range(3):
        assert torch.equal(_clip_check(grads, 1.0, False, ws), first)
    assert float(_clip([], [], 1.0, ws)) == 0.0
    zero = [torch.zeros(100, device="cuda")]
    assert float(_clip_check(zero, 1.0, False, ws)) == 0.0
    g = [_normal((1000,), 1.0, 1, torch.float32), _normal((500,), 1.0, 2)]
    g[1][77] = float("nan")
    outs = [torch.empty_like(t) for t in g]
    assert bool(torch.isnan(_clip(g, outs, 1.0, ws)).all())
    assert all(bool(torch.isnan(o).all()) for o in outs)
    g[1][77] = float("inf")
    assert bool(torch.isinf(_clip(g, outs, 1.0, ws)).all())
    assert bool((outs[0] == 0).all()) and bool(torch.isnan(outs[1][77]))


def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_moe_layer.py")
    spec = importlib.util.spec_from_file_location("train_moe_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_layer_gradients_against_autograd():
    """The example's layer against automatic differentiation in 64 bits with
    the same routing.  At most eight roundings to bf16, 2^-8 relative each at
    most, lie between an input and a gradient (h, a, expert_y, y; d_expert_y,
    dh, d_expert_x, d_x); to first order, and in norm, a gradient is off by no
    more than eight of them: 2^-5."""
    import combine_moe_dispatch_gb300 as moe
    N, H, I, E, K = 96, 128, 192, 8, 2
    layer = _example().MoELayer(N, H, I, E, K, seed=3)
    x = _normal((N, H), 1.0, 21)
    d_y = _normal((N, H), 0.1, 22)
    y = layer.forward(x).clone()
    d_x = layer.backward(d_y)
    assert moe.read_status(layer.b.workspace) == moe.Status.OK
    x64 = x.to(D).requires_grad_()
    ps = [p.to(D).requires_grad_() for p in layer.params]
    idx = layer.topk_idx.long()
    w = torch.softmax((x64 @ ps[0].t()).gather(1, idx), 1)
    want = torch.zeros((N, H), dtype=D, device="cuda")
    for k in range(K):
        gu = torch.einsum("nh,nfh->nf", x64, ps[1][idx[:, k]])
        a = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        want = want + w[:, k:k + 1] * torch.einsum("ni,nhi->nh", a, ps[2][idx[:, k]])
    want.backward(d_y.to(D))
    for got, ref, what in [(y, want.detach(), "y"), (d_x, x64.grad, "d_x"),
                           *[(g, p.grad, f"gradient {i}") for i, (g, p) in enumerate(zip(layer.grads, ps))]]:
        assert float((got.to(D) - ref).norm()) <= 2.0 ** -5 * float(ref.norm()), what


def test_example_learns():
    """A few clipped gradient steps of the example lower its loss, and every
    norm that it reports is the norm of its gradients."""
    layer = _example().MoELayer(128, 256, 256, 8, 2, seed=5)
    x, target = _normal((128, 256), 1.0, 31), _normal((128, 256), 1.0, 32, torch.float32)
    losses = []
    for _ in range(12):
        diff = layer.forward(x).float() - target
        losses.append(float(diff.square().mean()))
        layer.backward((diff / 128).bfloat16())
        norm = sum(float(g.to(D).square().sum()) for g in layer.grads) ** 0.5
        layer.step(lr=0.5, max_norm=1.0)
        assert abs(float(layer.grad_norm) - norm) <= 2.0 ** -16 * norm
    assert losses[-1] < losses[0]


def test_combine_backward_against_differences():
    """The loss sum(y * d_y), with y the weighted sum of the experts' rows and
    the weights the softmax of the chosen logits, moved by a small step along a
    random direction of the rows and of the logits, in 64 bits: the central
    differences agree with the gradients' inner products.  d_expert_y is off by
    one bf16 rounding (2^-8 relative) per element, d_logits by binary32
    roundings: 2^-8 and 2^-12 of the gradients' norms, times the direction's
    spread of a few, stay below the 2 % and 0.2 % asked."""
    import combine_moe_dispatch_gb300 as moe
    N, H, E, K = 24, 200, 10, 3
    shape = moe.make_shape(1, N, H, E, K, N)
    logits = _normal((N, E), 1.0, 41, torch.float32)
    idx = torch.empty((N, K), dtype=torch.int32, device="cuda")
    w = torch.empty((N, K), device="cuda")
    moe.router_topk(shape, logits, idx, w)
    b = moe.Buffers(shape, expert_x=False, expert_y=False)
    b.plan(idx)
    dy, ey = _normal((N, H), 1.0, 42), _normal((E, N, H), 1.0, 43)
    dey = torch.zeros((E, N, H), dtype=torch.bfloat16, device="cuda")
    dw, dl = torch.empty((N, K), device="cuda"), torch.empty((N, E), device="cuda")
    moe.combine_backward(shape, dy, ey, idx, b.slot_of, w, dey, dw, dl, b.workspace)
    e, s = idx.long(), b.slot_of.long()

    def loss(rows, logits):
        weights = torch.softmax(logits.gather(1, e), 1)
        return float(((weights[:, :, None] * rows[e, s]).sum(1) * dy.to(D)).sum())

    at, step = [ey.to(D), logits.to(D)], 1e-5
    for i, (grad, part) in enumerate(((dey, 0.02), (dl, 0.002))):
        v = torch.randn(at[i].shape, dtype=D, device="cuda", generator=_gen(50 + i))
        up = [t + step * v if j == i else t for j, t in enumerate(at)]
        down = [t - step * v if j == i else t for j, t in enumerate(at)]
        slope = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(float((grad.to(D) * v).sum()) - slope) <= part * float(grad.to(D).norm()), i


def test_offsets_past_32_bits():
    """Rows of the experts' buffers past 2^31 elements, and a gradient of more
    than 2^31 elements."""
    import combine_moe_dispatch_gb300 as moe
    N, H, E, cap = 4, 8192, 5, 65536
    shape = moe.make_shape(1, N, H, E, 1, cap)
    ws = torch.zeros(moe.workspace_size(shape), dtype=torch.uint8, device="cuda")
    idx = torch.full((N, 1), E - 1, dtype=torch.int32, device="cuda")
    slot = torch.arange(cap - N, cap, dtype=torch.int32, device="cuda")[:, None].contiguous()
    w = torch.full((N, 1), 0.5, device="cuda")
    dy = _normal((N, H), 1.0, 61)
    ey = torch.empty((E, cap, H), dtype=torch.bfloat16, device="cuda")
    ey[-1, -N:] = _normal((N, H), 1.0, 62)
    dey = torch.empty_like(ey)
    dey[-1, -2 * N:] = SENTINEL
    dw = torch.empty((N, 1), device="cuda")
    moe.combine_backward(shape, dy, ey, idx, slot, w, dey, dw, None, ws)
    assert torch.equal(dey[-1, -N:], (0.5 * dy.float()).bfloat16())
    assert bool((dey[-1, -2 * N:-N] == SENTINEL).all())
    terms = dy.to(D) * ey[-1, -N:].to(D)
    _near(dw[:, 0], terms.sum(1), H * U24 * terms.abs().sum(1), "d_weights")
    del ey, dey
    n = 2 ** 31 + 1001
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[2 ** 31 + 7], g[-1] = 3.0, 4.0, 12.0
    assert abs(float(_clip([g], [g], 6.5)) - 13.0) <= 2.0 ** -16 * 13.0
    for i, want in ((0, 1.5), (2 ** 31 + 7, 2.0), (n - 1, 6.0)):
        assert abs(float(g[i]) - want) <= (U8 + 2.0 ** -15) * want
    assert int((g != 0).sum()) == 3
