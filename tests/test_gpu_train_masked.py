"""moe_combine_backward where entries are left out after the router's softmax.

The forward pass is y = sum over the routed entries of w_k row_k with w the
softmax over all K chosen logits, so that the logit of an entry that is not
routed still has a derivative, -w_m sum_j w_j <dy, row_j>.

Tolerances: as for moe_combine_backward in general.  A dot product over H
elements in binary32 is off by at most H 2^-24 of the sum of its terms'
magnitudes; d_logits adds those errors, weighted, and K + 4 binary32
operations."""
import pytest
import torch

pytestmark = pytest.mark.gpu

D = torch.float64
U24 = 2.0 ** -24
SENTINEL = -12345.0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, std, seed, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=_gen(seed))


def _case(N, H, E, K, drop):
    """The step's plan with the dropped entries masked, and the routing as the
    router chose it."""
    import combine_moe_dispatch_gb300 as moe
    shape = moe.make_shape(1, N, H, E, K, N)
    logits = _normal((N, E), 1.0, 1, torch.float32)
    idx = torch.empty((N, K), dtype=torch.int32, device="cuda")
    w = torch.empty((N, K), device="cuda")
    moe.router_topk(shape, logits, idx, w)
    masked = torch.where(drop, -1, idx).int().contiguous()
    b = moe.Buffers(shape, expert_x=False, expert_y=False)
    b.plan_masked(masked)
    assert torch.equal(b.slot_of < 0, drop)
    dy, ey = _normal((N, H), 1.0, 2), _normal((E, N, H), 1.0, 3)
    for e, n in enumerate(b.expert_num_tokens.tolist()):
        ey[e, n:] = float("nan")
    out = [torch.full((E, N, H), SENTINEL, dtype=torch.bfloat16, device="cuda"),
           torch.full((N, K), SENTINEL, device="cuda"), torch.full((N, E), SENTINEL, device="cuda")]
    return moe, shape, logits, idx, masked, w, b, dy, ey, out


def _want(logits, idx, drop, slot, dy, ey):
    """d_weights and d_logits by automatic differentiation in 64 bits, and
    d_logits' tolerance."""
    N, K = idx.shape
    H = dy.shape[1]
    l64 = logits.to(D).requires_grad_()
    e = idx.long()
    w = torch.softmax(l64.gather(1, e), 1)
    rows = torch.where(drop[:, :, None], 0.0, ey[e, slot.clamp_min(0).long()].to(D))
    terms = rows * dy.to(D)[:, None, :]
    (w[:, :, None] * terms).sum().backward()
    w = w.detach()
    dw, tol = terms.sum(2), H * U24 * terms.abs().sum(2)
    spread = (w * (dw.abs() + tol)).sum(1, keepdim=True)
    # the weights of the call are binary32, one and a half units off at most: 3
    # times 2^-24 on the entry's own and on every one in the sum
    t = w * (tol + (w * tol).sum(1, keepdim=True) + (K + 10) * U24 * (dw.abs() + tol + spread))
    return dw, tol, l64.grad, torch.zeros_like(l64.grad).scatter_(1, e, t)


def _near(got, want, tol, what):
    bad = ~((got.to(D) - want).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off"


# one warp per token and eight, K above a group of 8, one token
SHAPES = [(1, 64, 8, 2), (45, 256, 16, 4), (20, 2056, 24, 8), (33, 512, 64, 11), (9, 4096, 40, 32)]


@pytest.mark.parametrize("N,H,E,K", SHAPES)
def test_logits_of_entries_left_out(N, H, E, K):
    """With the router's own choice in topk_idx, d_logits is the loss's
    derivative, the left-out entries' logits included; with -1 there, the
    same without those logits."""
    drop = torch.rand((N, K), device="cuda", generator=_gen(7)) < 0.4
    drop[0, 0], drop[0, 1] = True, False
    if N > 2:
        drop[N // 2] = True                    # nothing routed
    moe, shape, logits, idx, masked, w, b, dy, ey, (dey, dw, dl) = _case(N, H, E, K, drop)
    dw64, dw_tol, dl64, tol = _want(logits, idx, drop, b.slot_of, dy, ey)
    # weights of a token with nothing routed are not used
    w[drop.all(1)] = float("nan")
    moe.combine_backward(shape, dy, ey, idx, b.slot_of, w, dey, dw, dl, b.workspace)
    assert moe.read_status(b.workspace) == moe.Status.OK
    _near(dw, dw64, dw_tol, "d_weights")
    assert bool((dw[drop] == 0).all())
    _near(dl, dl64, tol, "d_logits")
    assert float(dl64.gather(1, idx.long())[drop].abs().max()) > 0.0       # they are not all 0
    for e, n in enumerate(b.expert_num_tokens.tolist()):
        assert bool((dey[e, n:] == SENTINEL).all()), "rows past the count were written"
    dl.fill_(SENTINEL)
    moe.combine_backward(shape, dy, ey, masked, b.slot_of, w, dey, dw, dl, b.workspace)
    gone = torch.zeros((N, E), device="cuda").scatter_(1, idx.long(), drop.float()) > 0
    _near(dl, torch.where(gone, 0.0, dl64), tol, "d_logits without the experts")


def test_chosen_twice_and_left_out_once():
    """An expert chosen twice, one of the entries left out: its logit gets the
    sum of both.  A weight of 0 (normalised over the routed entries) leaves 0."""
    N, H, E, K = 5, 128, 6, 3
    drop = torch.zeros((N, K), dtype=torch.bool, device="cuda")
    drop[:, 1] = True
    moe, shape, _, _, _, _, b, dy, ey, (dey, dw, dl) = _case(N, H, E, K, drop)
    idx = torch.tensor([[2, 2, 4]] * N, dtype=torch.int32, device="cuda")
    masked = torch.where(drop, -1, idx).int().contiguous()
    b.plan_masked(masked)
    ey = _normal((E, N, H), 1.0, 4)
    for share in (0.25, 0.0):
        w = torch.tensor([[0.5, share, 0.5 - share]] * N, device="cuda")
        moe.combine_backward(shape, dy, ey, idx, b.slot_of, w, dey, dw, dl, b.workspace)
        rows = ey[idx.long(), b.slot_of.clamp_min(0).long()].to(D)
        terms = torch.where(drop[:, :, None], 0.0, rows * dy.to(D)[:, None, :])
        dw64, mag = terms.sum(2), terms.abs().sum(2)
        own = w.to(D) * (dw64 - (w.to(D) * dw64).sum(1, keepdim=True))
        dl64 = torch.zeros((N, E), dtype=D, device="cuda").scatter_add_(1, idx.long(), own)
        _near(dl, dl64, torch.full_like(dl64, 4 * H * U24 * float(mag.max())), f"d_logits, share {share}")


@pytest.mark.parametrize("kind", ["expert", "negative expert", "slot", "negative slot"])
def test_entries_out_of_range(kind):
    """One entry out of range, in a batch that one block handles (so that no block
    starts after the error): it is skipped, its logit gets nothing and its row
    is not written, the status reports it, and every other entry is as without it."""
    N, H, E, K = 6, 64, 4, 3
    drop = torch.zeros((N, K), dtype=torch.bool, device="cuda")
    moe, shape, _, idx, _, w, b, dy, _, (dey, dw, dl) = _case(N, H, E, K, drop)
    ey = _normal((E, N, H), 1.0, 8)
    bad_idx, bad_slot, at = idx.clone(), b.slot_of.clone(), (2, 1)
    if kind.endswith("expert"):
        bad_idx[at] = -7 if "negative" in kind else E
    else:
        bad_slot[at] = -2 if "negative" in kind else N
    moe.combine_backward(shape, dy, ey, bad_idx, bad_slot, w, dey, dw, dl, b.workspace)
    assert moe.read_status(b.workspace) == (moe.Status.BAD_EXPERT if kind.endswith("expert") else
                                            moe.Status.CAPACITY)
    ok = torch.ones((N, K), dtype=torch.bool, device="cuda")
    ok[at] = False
    e, s = idx.long(), b.slot_of.long()
    assert bool((dey[e[at], s[at]] == SENTINEL).all())
    want = w.to(D)[:, :, None] * dy.to(D)[:, None, :]
    got = dey[e, s].to(D)
    assert bool(((got - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs())[ok].all())
    terms = torch.where(ok[:, :, None], ey[e, s].to(D) * dy.to(D)[:, None, :], 0.0)
    dw64, dw_tol = terms.sum(2), H * U24 * terms.abs().sum(2)
    _near(dw, dw64, dw_tol, "d_weights")
    w64 = torch.where(ok, w.to(D), 0.0)
    own = w64 * (dw64 - (w64 * dw64).sum(1, keepdim=True))
    spread = (w64 * (dw64.abs() + dw_tol)).sum(1, keepdim=True)
    tol = w64 * (dw_tol + (w64 * dw_tol).sum(1, keepdim=True) + (K + 4) * U24 * (dw64.abs() + dw_tol + spread))
    zero = torch.zeros((N, E), dtype=D, device="cuda")
    _near(dl, zero.scatter(1, e, own), zero.scatter(1, e, tol), "d_logits")
