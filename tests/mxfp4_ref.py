"""MXFP4 as the format defines it, in 64 bits: values, codes, and the places of
the scale bytes.  Used by the tests of the 4-bit operators."""
import torch

D = torch.float64
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def power(exponent):
    """2^exponent in 64 bits, exact."""
    return ((exponent.to(torch.int64) + 1023) << 52).view(D)


def quantise(v):
    """[..., cols] -> codes [..., cols] and biased exponents [..., cols/32].
    Nearest E2M1, ties to the even code, by comparison with every border."""
    b = v.to(D).reshape(*v.shape[:-1], -1, 32)
    bad = ~b.isfinite().all(-1)
    amax = torch.where(b.isfinite(), b, 0.0).abs().amax(-1)
    biased = torch.where(amax > 0, torch.frexp(amax).exponent - 3 + 127, 0).clamp(min=0)
    m = b.abs() / power(biased - 127)[..., None]
    code = torch.zeros(b.shape, dtype=torch.int64, device=v.device)
    for k in range(7):
        border = (GRID[k] + GRID[k + 1]) / 2
        code += (m > border) | ((m == border) & (k % 2 == 1))
    code += 8 * torch.signbit(b)
    code = torch.where(bad[..., None], 0, code)
    return code.reshape(v.shape), torch.where(bad, 255, biased)


def values(code, biased):
    """What codes and biased exponents stand for, in 64 bits."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=D, device=code.device)
    x = torch.where(biased == 255, float("nan"), power(biased - 127))
    return grid[code] * x.repeat_interleave(32, -1)


def pack(code):
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)


def unpack(q):
    q = q.to(torch.int64)
    return torch.stack([q % 16, q // 16], -1).reshape(*q.shape[:-1], -1)


def places(rows, cols, gate_up, device):
    """Where the scale of (row, block) stands among an expert's bytes."""
    r = torch.arange(rows, device=device)
    if gate_up:
        f, up = r % (rows // 2), r // (rows // 2)
        r = f // 64 * 128 + 64 * up + f % 64
    b = torch.arange(cols // 32, device=device)
    tiles = (cols + 127) // 128
    return ((r // 128 * tiles)[:, None] + b // 4) * 512 + (r % 32 * 16 + r % 128 // 32 * 4)[:, None] + b % 4


def scale_tensor(E, rows, cols, fill, device="cuda"):
    return torch.full((E, (rows + 127) // 128, (cols + 127) // 128, 512), fill, dtype=torch.uint8,
                      device=device)


def place(biased, scale, gate_up=False):
    """Write biased exponents [E, rows, blocks] into a scale tensor."""
    E, rows, nb = biased.shape
    at = places(rows, nb * 32, gate_up, biased.device)
    scale.view(E, -1)[:, at.reshape(-1)] = biased.reshape(E, -1).to(torch.uint8)
    return scale


def take(scale, rows, cols, gate_up=False):
    E = scale.shape[0]
    at = places(rows, cols, gate_up, scale.device)
    return scale.view(E, -1)[:, at.reshape(-1)].view(E, rows, cols // 32).to(torch.int64)
