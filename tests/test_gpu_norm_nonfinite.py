"""moe_add_rms_norm's E4M3 output of rows that are not finite: a block with a
NaN among its y reads back as NaN, scale and bytes, as the bf16 output of the
same call does; a block with an infinite y is not finite either; every other
block has the bytes of a call without such rows.  No tolerance: bytes and bits
are compared."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# H: every number of warps a row takes, a short last block, rows that do not fit the registers
WIDTHS = [16, 256, 272, 512, 1024, 1040, 2048, 4096, 7168, 8208, 16400]


def _rand(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g).bfloat16()


def _run(x, residual, gain, payload, with_y):
    """bf16 y, bytes and scales [N, nb] of the 8-bit output."""
    import combine_moe_dispatch_gb300 as moe
    N, H = x.shape
    nb = (H + 127) // 128
    y = torch.full_like(x, -7.0) if with_y else None
    q = torch.full((N, H), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((nb, N) if payload == moe.PAYLOAD_FP8_E4M3_TSCALE else (N, nb), -7.0, device="cuda")
    moe.add_rms_norm(moe.make_shape(1, N, H, 1, 1, 1, payload), x, residual, gain, 1e-6, None, y, q, scale)
    return y, q, scale.t() if payload == moe.PAYLOAD_FP8_E4M3_TSCALE else scale


def _blocks(t, fill):
    """[N, H] -> [N, nb, 128], the short last block filled up."""
    N, H = t.shape
    return torch.nn.functional.pad(t, (0, -H % 128), value=fill).view(N, -1, 128)


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("payload", [1, 2])
@pytest.mark.parametrize("residual", [False, True])
def test_non_finite_rows(H, payload, residual):
    import combine_moe_dispatch_gb300 as moe
    N = 21
    x, gain = _rand((N, H), 1), _rand((H,), 2)
    r = _rand((N, H), 3) if residual else None
    _, q0, scale0 = _run(x, r, gain, payload, True)
    x[2, H - 1], x[7, 0], x[8, H // 2], x[19] = float("nan"), float("inf"), float("-inf"), float("nan")
    if residual:
        r[11, 3], x[13, 5], r[13, 5] = float("nan"), float("inf"), float("-inf")
    y = torch.empty_like(x)
    moe.add_rms_norm(moe.make_shape(1, N, H, 1, 1, 1), x, r, gain, 1e-6, None, y)
    nan = _blocks(y, 0.0).isnan().any(-1)
    assert bool(nan[2].all()) and bool(nan[19].all()) and int(nan[7].sum()) == 1 and int(nan[8].sum()) == 1
    infinite = {7, 8}
    for with_y in (True, False):
        y8, q, scale = _run(x, r, gain, payload, with_y)
        if with_y:
            assert torch.equal(y8.view(torch.int16), y.view(torch.int16))
        assert torch.equal(scale.isnan(), nan)
        blocks = _blocks(q, 0x7F)
        assert bool((blocks[nan] & 0x7F == 0x7F).all())
        for i in range(N):
            if i in infinite:                # 1 / rms is 0: the other blocks are
                assert bool((blocks[i][~nan[i]] & 0x7F == torch.where(
                    _blocks(torch.ones_like(q), 0)[i][~nan[i]] > 0, 0, 0x7F)).all())
                assert bool((scale[i][~nan[i]] == 0.0).all())
            elif not bool(nan[i].any()):
                assert torch.equal(q[i], q0[i]) and torch.equal(scale[i], scale0[i])


@pytest.mark.parametrize("payload", [1, 2])
def test_non_finite_gain(payload):
    """A column's gain of NaN poisons that column's block in every row; one whose
    product passes binary32 leaves its block without a finite number."""
    N, H = 9, 656
    x, gain = _rand((N, H), 4), _rand((H,), 5)
    x[:, 300] = 3.0
    x[4] = 0.0
    _, q0, scale0 = _run(x, None, gain, payload, True)
    gain[130], gain[300] = float("nan"), 3.3e38
    y, q, scale = _run(x, None, gain, payload, True)
    assert bool(scale[:, 1].isnan().all()) and bool((q[:, 128:256] & 0x7F == 0x7F).all())
    rows = [i for i in range(N) if i != 4]
    value = q.view(torch.float8_e4m3fn).double() * scale.double().repeat_interleave(128, 1)[:, :H]
    assert bool(y[rows, 300].isinf().all()) and bool(value[rows, 256:384].isnan().all())
    assert bool((value[4, 256:384] == 0.0).all())
    for b in (0, 3, 4, 5):
        cut = slice(128 * b, 128 * b + 128)
        assert torch.equal(q[:, cut], q0[:, cut]) and torch.equal(scale[:, b], scale0[:, b])
