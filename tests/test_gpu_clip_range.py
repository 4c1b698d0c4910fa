"""moe_clip_grad_norm of gradients whose squares binary32 does not hold.

Tolerances as for the norm in general: binary32 over at most 64 squares (2^-24
each, half of it through the root) and one rounding, below 2^-16 relative;
the clipped values add three binary32 operations and the rounding to their type."""
import pytest
import torch

pytestmark = pytest.mark.gpu

D = torch.float64


def _normal(n, std, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.empty(n, dtype=D, device="cuda").normal_(0.0, 1.0, generator=g) * std).to(dtype)


def _check(grads, max_norm):
    import combine_moe_dispatch_gb300 as moe
    ws = torch.zeros(moe.clip_workspace_size(), dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    outs = [torch.empty_like(g) for g in grads]
    moe.clip_grad_norm(grads, outs, max_norm, norm, ws)
    want = sum(float(g.to(D).square().sum()) for g in grads) ** 0.5
    assert abs(float(norm) - want) <= 2.0 ** -16 * want, (float(norm), want)
    coef = min(1.0, max_norm / (want + 1e-6))
    for o, g in zip(outs, grads):
        u = 2.0 ** -24 if g.dtype == torch.float32 else 2.0 ** -8
        ref = g.to(D) * coef
        # + the last place of a subnormal result
        assert bool(((o.to(D) - ref).abs() <= (u + 2.0 ** -15) * ref.abs() + 2.0 ** -133).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("std", [1e-37, 1e-30, 1e-22, 1e-13, 1e-6, 1e10, 1e18, 1e20, 1e30, 1e34])
@pytest.mark.parametrize("n", [1, 9, 16384, 200001])
def test_any_scale(dtype, std, n):
    _check([_normal(n, std, 1, dtype)], 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scales_together(dtype):
    """One huge value among ordinary ones, tiny ones beside zeros, and a tensor of
    zeros, at odd addresses."""
    big = _normal(100003, 1.0, 2, dtype)
    big[70001] = 1e25
    few = torch.zeros(50000, dtype=dtype, device="cuda")
    few[12345] = 1e-25
    zeros = torch.zeros(300000, dtype=dtype, device="cuda")
    _check([big[1:], few[3:], zeros], 10.0)
    _check([few[3:], zeros[1:]], 10.0)
    _check([few[3:], -zeros, _normal(70, 1e-3, 3, dtype)], 1e-4)
