"""Cases that measure the operators of a Mixture-of-Experts block served in 4
bits: the root-mean-square norm before it (with the residual's addition, an
output in 8 bits, and its backward pass), quantisation to MXFP4 and back, the
dispatch that quantises, and the experts' feed-forward on 4-bit operands.

``run`` computes an operator either through this package's entry points
(``own`` true) or in its plain form: elementary torch operations in 32 bits,
rounded once at the end.  ``exact`` is the definition in 64 bits.

MXFP4 (OCP Microscaling Formats 1.0): blocks of 32 elements of a row share the
power of two X = 2^(floor(log2 amax) - 2), held as its biased exponent in a
byte; an element is the E2M1 number nearest to x / X (ties to even, at most 6 in
magnitude), two to a byte, the earlier one in the low half.  The scale bytes
of an array of rows stand in tiles of 128 rows x 4 blocks, row r and block b of
a tile at 16 (r mod 32) + 4 (r / 32) + b; the tiles of the gate and up weights
hold 64 rows of the gate, then the same 64 of up.

Notation: E experts, cap rows per expert, H hidden size, I intermediate size,
N tokens with K experts each.  Expert e has count[e] <= cap rows; rows from
count[e] on are never read (their scales are NaN here) and never written.
"""
import random

import numpy as np
import torch

own = False

EPS = 1e-6
MAX_FFN_FLOPS = 2.7e12        # largest work of one drawn feed-forward
MAX_ROW_ELEMENTS = 58_000_000  # and of the other operators' rows
POOL_BLOCKS = 1_048_583       # a prime number of blocks: repeated, no two rows line up


# --- the cases ---------------------------------------------------------------

def listed():
    return [
        # One token of a Mixtral-shaped layer, between two layers: latency.
        dict(name="norm_one_token", op="norm", N=1, H=4096, residual=True, fp8=False),
        # A prompt's tokens of a DeepSeek-V3-shaped layer, with the 8-bit rows for
        # the products that take them: bound by memory.
        dict(name="norm_prefill", op="norm", N=8192, H=7168, residual=True, fp8=True),
        # Training of a small layer whose sizes fit no tile.
        dict(name="norm_bwd_odd", op="norm_bwd", N=333, H=264, d_sum=False),
        # Training batch: the gradient also comes along the residual stream.
        dict(name="norm_bwd_batch", op="norm_bwd", N=8192, H=7168, d_sum=True),
        # The shared expert's rows of a decode step, quantised and read back.
        dict(name="quant_rows", op="quant", E=1, rows=1024, cols=7168, gate_up=False),
        # A Mixtral-shaped layer's gate and up weights, prepared for serving.
        dict(name="quant_weights", op="quant", E=8, rows=28672, cols=4096, gate_up=True),
        # Dispatch of the tiny layer: latency.
        dict(name="dispatch_tiny", op="dispatch", N=64, K=2, E=8, cap=64, H=256, masked=0.1),
        # DeepSeek-V3-shaped decode step: 1024 tokens to 8 of 256 experts.
        dict(name="dispatch_decode", op="dispatch", N=1024, K=8, E=256, cap=128, H=7168, masked=0.0),
        # One token of a Mixtral-shaped layer: the weights of two experts once.
        dict(name="ffn_one_token", op="ffn", E=8, cap=1, H=4096, I=14336, rows=2, skew=0.0, draw=1),
        # Small and odd: no size is a multiple of any tile, one expert is empty.
        dict(name="ffn_odd", op="ffn", E=5, cap=37, H=288, I=160, rows=61, skew=0.8, draw=2),
        # DeepSeek-V3-shaped decode step, about 32 rows an expert: 6 GB of weights.
        dict(name="ffn_decode", op="ffn", E=256, cap=128, H=7168, I=2048, rows=8192, skew=0.0, draw=3),
        # Mixtral-shaped layer, 8 x 512 tokens, top-2: bound by the tensor cores.
        dict(name="ffn_batch", op="ffn", E=8, cap=2048, H=4096, I=14336, rows=8192, skew=0.0, draw=4),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(lo * (hi / lo) ** rng.random() / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant", "dispatch", "ffn", "ffn"])
    while op in ("norm", "norm_bwd"):
        N, H = _log_int(rng, 1, 8192), _log_int(rng, 64, 7168, 16 if op == "norm" else 8)
        if N * H < MAX_ROW_ELEMENTS:
            if op == "norm":
                return dict(op=op, N=N, H=H, residual=rng.random() < 0.7, fp8=rng.random() < 0.5)
            return dict(op=op, N=N, H=H, d_sum=rng.random() < 0.5)
    while op == "quant":
        E, rows, cols = _log_int(rng, 1, 64), _log_int(rng, 1, 28672), _log_int(rng, 32, 14336, 32)
        gate_up = rows % 2 == 0 and rng.random() < 0.5
        if E * rows * cols < 900_000_000:
            return dict(op=op, E=E, rows=rows, cols=cols, gate_up=gate_up)
    while op == "dispatch":
        N, E, H = _log_int(rng, 1, 4096), _log_int(rng, 2, 384), _log_int(rng, 64, 7168, 32)
        K = min(E, rng.choice([1, 2, 4, 6, 8]))
        if N * K * H < MAX_ROW_ELEMENTS:
            return dict(op=op, N=N, K=K, E=E, cap=min(N, int(2.0 * N * K / E) + 24), H=H,
                        masked=rng.choice([0.0, 0.1, 0.5]))
    while True:
        E, H, I = _log_int(rng, 1, 256), _log_int(rng, 128, 7168, 32), _log_int(rng, 128, 14336, 32)
        rows, skew = _log_int(rng, 1, 8192), rng.choice([0.0, 0.0, 0.5, 1.0])
        cap = min(rows, max(4, int(rows / E * (1.5 if skew == 0.0 else 4.0)) + 16))
        if (6.0 * rows * H * I < MAX_FFN_FLOPS and 6.0 * E * cap * H * I < 2 * MAX_FFN_FLOPS and
                3 * E * H * I < 6e9):
            return dict(op=op, E=E, cap=cap, H=H, I=I, rows=rows, skew=skew,
                        draw=rng.randrange(1 << 20))


# --- inputs ------------------------------------------------------------------

def _counts(case):
    """Rows per expert, as the routing leaves them: `rows` draws over the
    experts with popularity 1/j^skew, what passes `cap` moved on to experts
    with room.  They depend on the case alone; a seed permutes them."""
    E, cap = case["E"], case["cap"]
    rng = np.random.default_rng(case["draw"])
    p = 1.0 / np.arange(1, E + 1) ** case["skew"]
    counts = rng.multinomial(min(case["rows"], E * cap), p / p.sum())
    over = int(np.maximum(counts - cap, 0).sum())
    counts = np.minimum(counts, cap)
    for e in np.argsort(-counts, kind="stable"):
        add = min(over, cap - counts[e])
        counts[e] += add
        over -= add
    if E > 2 and case["skew"] > 0.0:          # skewed routing leaves some expert empty
        counts[E - 1] = 0
    return counts


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, std, g, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _rows(shape, g):
    """Hidden states: normal, rows and some columns of different magnitude."""
    t = _normal(shape, 1.0, g, torch.float32)
    t *= torch.exp(_normal(shape[:-1] + (1,), 0.5, g, torch.float32))
    t *= torch.exp(_normal(shape[-1:], 0.5, g, torch.float32))
    return t.to(torch.bfloat16)


def _power(biased):
    """2^(biased - 127) in 32 bits; 255 is NaN."""
    bits = torch.where(biased > 0, biased << 23, torch.full_like(biased, 1 << 22))
    return torch.where(biased == 255, float("nan"), bits.view(torch.float32))


def _quantise(v):
    """Values [..., 32] in 32 bits -> E2M1 values and biased exponents."""
    biased = (v.abs().amax(-1).view(torch.int32) >> 23) - 2      # of X, from the largest magnitude
    biased = biased.clamp(min=0)
    t = v * _power(254 - biased)[..., None]
    m = t.abs()
    q = torch.where(m < 2.0, torch.round(m * 2.0) * 0.5,
                    torch.where(m < 4.0, torch.round(m), torch.round(m * 0.5) * 2.0)).clamp(max=6.0)
    return torch.copysign(q, t), biased


def _codes(q):
    """E2M1 values -> packed bytes."""
    m = (q.abs() * 2.0).to(torch.int32)                           # 0 1 2 3 4 6 8 12
    code = torch.where(m < 4, m, torch.where(m < 8, 4 + (m - 4) // 2, 6 + (m - 8) // 4))
    code = (code + 8 * torch.signbit(q)).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _tiled(scale, gate_up):
    """Scale bytes [E, rows, blocks] -> tiles [E, row tiles, block tiles, 512]."""
    E, rows, nb = scale.shape
    pad = torch.nn.functional.pad
    if gate_up:
        scale = pad(scale.view(E, 2, rows // 2, nb), (0, 0, 0, -(rows // 2) % 64))
        scale = scale.view(E, 2, -1, 64, nb).transpose(1, 2).reshape(E, -1, nb)
    scale = pad(scale, (0, -nb % 4, 0, -scale.shape[1] % 128))
    t = scale.view(E, scale.shape[1] // 128, 4, 32, scale.shape[2] // 4, 4)
    return t.permute(0, 1, 4, 3, 2, 5).reshape(E, t.shape[1], t.shape[4], 512).contiguous()


def _untiled(tiles, rows, blocks, gate_up):
    """The other way."""
    E, rt, bt, _ = tiles.shape
    t = tiles.view(E, rt, bt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, rt * 128, bt * 4)
    if gate_up:
        t = t.view(E, rt, 2, 64, bt * 4).transpose(1, 2).reshape(E, 2, rt * 64, bt * 4)
        t = t[:, :, :rows // 2].reshape(E, rows, bt * 4)
    return t[:, :rows, :blocks]


def _weights(E, rows, cols, std, g, gate_up=False):
    """Quantised normal weights: a pool of blocks, repeated."""
    q, biased = _quantise(_normal((POOL_BLOCKS, 32), std, g, torch.float32))
    packed, biased = _codes(q), biased.to(torch.uint8)
    n = E * rows * cols // 32
    times = -(-n // POOL_BLOCKS)
    return (packed.repeat(times, 1)[:n].reshape(E, rows, cols // 2),
            _tiled(biased.repeat(times)[:n].reshape(E, rows, cols // 32), gate_up))


def _routing(case, g):
    N, K, E, cap = case["N"], case["K"], case["E"], case["cap"]
    idx = torch.rand((N, E), device="cuda", generator=g).argsort(1)[:, :K].contiguous()
    idx[torch.rand((N, K), device="cuda", generator=g) < case["masked"]] = -1
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    first = torch.searchsorted(flat[order].contiguous(), flat)
    slot = torch.empty_like(flat)
    slot[order] = torch.arange(N * K, device="cuda")
    slot = slot - first
    out = (flat < 0) | (slot >= cap)          # not routed, or dropped at capacity
    slot[out] = -1
    flat = torch.where(out, torch.full_like(flat, -1), flat)
    counts = torch.bincount(flat[~out], minlength=E)
    return flat.reshape(N, K).int(), slot.reshape(N, K).int(), counts.int()


def _tiles(E, rows, cols):
    return torch.zeros((E, -(-rows // 128), -(-cols // 128), 512), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g, op, bf16 = _gen(seed), case["op"], torch.bfloat16
    zeros = lambda dims, dt: torch.zeros(dims, dtype=dt, device="cuda")  # noqa: E731
    s = dict(case=case)
    if op in ("norm", "norm_bwd"):
        N, H = case["N"], case["H"]
        s["gain"] = (1.0 + _normal((H,), 0.2, g, torch.float32)).to(bf16)
        s["x"] = _rows((N, H), g)
        if op == "norm":
            s["residual"] = _rows((N, H), g) if case["residual"] else None
            s["sum"] = zeros((N, H), bf16) if case["residual"] else None
            s["y"] = zeros((N, H), bf16)
            s["y_q"] = zeros((N, H), torch.uint8) if case["fp8"] else None
            s["y_scale"] = zeros((N, -(-H // 128)), torch.float32) if case["fp8"] else None
        else:
            s["d_y"] = _normal((N, H), 0.1, g)
            s["d_sum"] = _normal((N, H), 0.1, g) if case["d_sum"] else None
            s["d_x"] = zeros((N, H), bf16)
            s["d_gain"] = zeros((H,), torch.float32)
        if own:
            import combine_moe_dispatch_gb300 as moe
            payload = moe.PAYLOAD_FP8_E4M3 if case.get("fp8") else moe.PAYLOAD_BF16
            s["shape"] = moe.make_shape(1, N, H, 1, 1, 1, payload)
            if op == "norm_bwd":
                s["workspace"] = zeros((moe.norm_workspace_size(s["shape"]),), torch.uint8)
        return s
    if op == "quant":
        E, rows, cols = case["E"], case["rows"], case["cols"]
        s["src"] = torch.empty((E, rows, cols), dtype=bf16, device="cuda")
        for e in range(E):
            s["src"][e] = _rows((rows, cols), g)
        s["q"] = zeros((E, rows, cols // 2), torch.uint8)
        s["scale"] = _tiles(E, rows, cols)
        s["out"] = torch.empty_like(s["src"])
        return s
    E, cap, H = case["E"], case["cap"], case["H"]
    if op == "dispatch":
        s["x"] = _rows((case["N"], H), g)
        s["topk_idx"], s["slot_of"], s["counts"] = _routing(case, g)
        s["expert_x"], s["expert_x_scale"] = zeros((E, cap, H // 2), torch.uint8), _tiles(E, cap, H)
        s["out"] = zeros((E, cap, H), bf16)
        if own:
            import combine_moe_dispatch_gb300 as moe
            s["shape"] = moe.make_shape(1, case["N"], H, E, case["K"], cap)
            s["workspace"] = zeros((moe.workspace_size(s["shape"]),), torch.uint8)
        return s
    I = case["I"]
    counts = np.random.default_rng(int(seed)).permutation(_counts(case)).astype(np.int32)
    s["counts"] = torch.from_numpy(counts).cuda()
    q, biased = _quantise(_rows((E, cap, H), g).float().view(E, cap, H // 32, 32))
    past = torch.arange(cap, device="cuda")[None, :] >= s["counts"][:, None]
    biased[past] = 255                                    # NaN
    s["expert_x"] = _codes(q).view(E, cap, H // 2)
    s["expert_x_scale"] = _tiled(biased.to(torch.uint8), False)
    s["w_gate_up"], s["w_gate_up_scale"] = _weights(E, 2 * I, H, H ** -0.5, g, True)
    s["w_down"], s["w_down_scale"] = _weights(E, H, I, I ** -0.5, g)
    s["expert_act"], s["expert_act_scale"] = zeros((E, cap, I // 2), torch.uint8), _tiles(E, cap, I)
    s["expert_y"] = zeros((E, cap, H), bf16)
    if own:
        import combine_moe_dispatch_gb300 as moe
        s["shape"] = moe.make_shape(1, max(1, case["rows"]), H, E, 1, cap)
        s["workspace"] = zeros((moe.ffn_mxfp4_workspace_size(s["shape"], I),), torch.uint8)
    return s


# --- one pass ----------------------------------------------------------------

def _run_own(s):
    import combine_moe_dispatch_gb300 as moe
    case = s["case"]
    op = case["op"]
    if op == "norm":
        moe.add_rms_norm(s["shape"], s["x"], s["residual"], s["gain"], EPS, s["sum"], s["y"],
                         s["y_q"], s["y_scale"])
        fp8 = [s["y_q"].view(torch.float8_e4m3fn), s["y_scale"]] if case["fp8"] else []
        return [s["y"]] + ([s["sum"]] if case["residual"] else []) + fp8
    if op == "norm_bwd":
        moe.add_rms_norm_backward(s["shape"], s["d_y"], s["d_sum"], s["x"], s["gain"], EPS, s["d_x"],
                                  s["d_gain"], s["workspace"])
        return [s["d_x"], s["d_gain"]]
    if op == "quant":
        flags = moe.MXFP4_GATE_UP if case["gate_up"] else 0
        moe.quant_mxfp4(s["src"], None, s["q"], s["scale"], flags)
        moe.dequant_mxfp4(s["q"], s["scale"], None, s["out"], flags)
        return [s["out"]]
    if op == "dispatch":
        moe.dispatch_mxfp4(s["shape"], s["x"], s["topk_idx"], s["slot_of"], s["expert_x"],
                           s["expert_x_scale"], s["workspace"])
        moe.dequant_mxfp4(s["expert_x"], s["expert_x_scale"], s["counts"], s["out"])
        return [s["out"]]
    moe.ffn_mxfp4(s["shape"], case["I"], s["expert_x"], s["expert_x_scale"], s["w_gate_up"],
                  s["w_gate_up_scale"], s["w_down"], s["w_down_scale"], s["counts"], s["expert_act"],
                  s["expert_act_scale"], s["expert_y"], s["workspace"])
    return [s["expert_y"]]


def _values(packed, tiles, gate_up):
    """What 4-bit rows stand for, in 32 bits."""
    E, rows, half = packed.shape
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    table = torch.cat([table, -table])
    byte = torch.arange(256, device="cuda")
    pairs = torch.stack([table[byte & 15], table[byte >> 4]], 1)
    v = torch.nn.functional.embedding(packed.int(), pairs).view(E, rows, half // 16, 32)
    power = _power(_untiled(tiles, rows, half // 16, gate_up).int())
    return v.mul_(power[..., None]).view(E, rows, half * 2)


def _plain_norm(s):
    case, bf16 = s["case"], torch.bfloat16
    row = s["x"].float()
    if case["residual"]:
        row = (row + s["residual"].float()).to(bf16).float()
    y = row * torch.rsqrt(row.square().mean(1, keepdim=True) + EPS) * s["gain"].float()
    out = [y.to(bf16)] + ([row.to(bf16)] if case["residual"] else [])
    if case["fp8"]:
        N, H = y.shape
        blocks = torch.nn.functional.pad(y, (0, -H % 128)).view(N, -1, 128)
        scale = blocks.abs().amax(2) / 448.0
        q = blocks / torch.where(scale > 0.0, scale, torch.ones_like(scale))[:, :, None]
        q = q.clamp(-448.0, 448.0).view(N, -1)[:, :H]
        out += [q.to(torch.float8_e4m3fn), scale]
    return out


def _plain_norm_bwd(s):
    row, dy, gain = s["x"].float(), s["d_y"].float(), s["gain"].float()
    rstd = torch.rsqrt(row.square().mean(1, keepdim=True) + EPS)
    u, g = row * rstd, dy * gain
    d_x = rstd * (g - u * (g * u).mean(1, keepdim=True))
    if s["d_sum"] is not None:
        d_x = d_x + s["d_sum"].float()
    return [d_x.to(torch.bfloat16), (dy * u).sum(0)]


def _plain_quant(s):
    src = s["src"]
    q, biased = _quantise(src.float().view(*src.shape[:2], -1, 32))
    v = q * _power(biased)[..., None]
    return [v.view(src.shape).to(torch.bfloat16)]


def _plain_dispatch(s):
    E, cap, H = s["out"].shape
    q, biased = _quantise(s["x"].float().view(-1, H // 32, 32))
    v = q * _power(biased)[..., None]
    v = v.view(-1, H).to(torch.bfloat16)
    routed = s["slot_of"] >= 0
    row = (s["topk_idx"] * cap + s["slot_of"]).long()[routed]
    token = torch.arange(len(v), device="cuda")[:, None].expand(routed.shape)[routed]
    out = torch.zeros((E * cap, H), dtype=torch.bfloat16, device="cuda")
    out[row] = v[token]
    return [out.view(E, cap, H)]


def _plain_ffn(s):
    E, cap, H = s["expert_y"].shape
    I = s["case"]["I"]
    below = (torch.arange(cap, device="cuda")[None, :] < s["counts"][:, None])[:, :, None]
    x = _values(s["expert_x"], s["expert_x_scale"], False)
    x = torch.where(below, x, torch.zeros((), device="cuda"))
    h = torch.bmm(x, _values(s["w_gate_up"], s["w_gate_up_scale"], True).transpose(1, 2))
    gate, up = h[:, :, :I], h[:, :, I:]
    q, biased = _quantise((gate / (1.0 + torch.exp(-gate)) * up).view(E, cap, I // 32, 32))
    a = (q * _power(biased)[..., None]).view(E, cap, I)
    y = torch.bmm(a, _values(s["w_down"], s["w_down_scale"], False).transpose(1, 2))
    return [y.to(torch.bfloat16)]


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "quant": _plain_quant,
         "dispatch": _plain_dispatch, "ffn": _plain_ffn}


def run(s):
    return _run_own(s) if own else PLAIN[s["case"]["op"]](s)


# --- what a pass cannot do without --------------------------------------------

FOUR_BITS = 17.0 / 32.0       # bytes of an element with its share of the scale


def work(case):
    op = case["op"]
    if op == "norm":
        N, H = case["N"], case["H"]
        arrays = 2 + (2 if case["residual"] else 0)
        fp8 = N * (H + 4 * -(-H // 128)) if case["fp8"] else 0
        return {"bytes": 2 * arrays * N * H + fp8 + 2 * H, "flops": 6.0 * N * H}
    if op == "norm_bwd":
        N, H = case["N"], case["H"]
        return {"bytes": (8 if case["d_sum"] else 6) * N * H + 6 * H, "flops": 12.0 * N * H}
    if op == "quant":
        n = case["E"] * case["rows"] * case["cols"]
        return {"bytes": n * (4 + 2 * FOUR_BITS), "flops": 4.0 * n}
    if op == "dispatch":
        N, K, H = case["N"], case["K"], case["H"]
        rows = N * K * (1.0 - case["masked"])
        return {"bytes": 2 * N * H + 8 * N * K + rows * H * (2 + 2 * FOUR_BITS), "flops": 3.0 * N * H}
    counts = _counts(case)
    rows, active, H, I = int(counts.sum()), int((counts > 0).sum()), case["H"], case["I"]
    return {"bytes": active * 3 * H * I * FOUR_BITS + rows * H * (2 + FOUR_BITS),
            "flops": 6.0 * rows * H * I}


# --- the definition in 64 bits -------------------------------------------------

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _two_to(exponent):
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _nearest(v):
    """MXFP4's values of v [..., 32] in 64 bits, by the borders between the
    E2M1 numbers (a tie goes to the one whose last bit is 0)."""
    exponent = torch.frexp(v.abs().amax(-1, keepdim=True)).exponent - 3
    power = _two_to(exponent.clamp(min=-127))
    m = v.abs() / power
    code = torch.zeros_like(m)
    for k in range(7):
        border = (E2M1[k] + E2M1[k + 1]) / 2
        code += (m >= border) if k % 2 else (m > border)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    return torch.copysign(grid[code.long()], v) * power


def _decode(packed, tiles, e, rows, gate_up):
    """Rows [0, rows) of expert e in 64 bits, each scale found by its place."""
    n, half = packed.shape[1], packed.shape[2]
    grid = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")
    b = packed[e, :rows].long()
    v = torch.stack([grid[b % 16], grid[b // 16]], 2).view(rows, half * 2)
    r = torch.arange(rows, device="cuda")
    if gate_up:
        f, up = r % (n // 2), r // (n // 2)
        r = (f // 64) * 128 + up * 64 + f % 64
    k = torch.arange(half // 16, device="cuda")
    at = 16 * (r % 32) + 4 * (r % 128 // 32)
    scale = tiles[e][(r // 128)[:, None], (k // 4)[None, :], at[:, None] + (k % 4)[None, :]]
    return v * _two_to(scale.long() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s, d, op = prepare(case, seed), torch.float64, case["op"]
    if op in ("norm", "norm_bwd"):
        outs = []
        d_gain = torch.zeros(case["H"], dtype=d, device="cuda")
        for a in range(0, case["N"], 1024):
            b = slice(a, a + 1024)
            row, gain = s["x"][b].to(d), s["gain"].to(d)
            if op == "norm":
                if case["residual"]:
                    row = (row + s["residual"][b].to(d)).to(torch.bfloat16).to(d)
                y = torch.nn.functional.rms_norm(row, (case["H"],), gain, EPS)
                part = [y] + ([row] if case["residual"] else [])
                if case["fp8"]:
                    cut = y.split(128, 1)
                    amax = torch.stack([c.abs().amax(1) for c in cut], 1)
                    div = torch.where(amax > 0, amax / 448.0, 1.0)
                    part += [torch.cat([c / div[:, i:i + 1] for i, c in enumerate(cut)], 1), amax / 448.0]
                outs.append(part)
                continue
            dy = s["d_y"][b].to(d)
            mean = (row * row).sum(1, keepdim=True) / case["H"] + EPS
            dot = (dy * gain * row).sum(1, keepdim=True) / case["H"]
            d_x = dy * gain / mean.sqrt() - row * dot / mean ** 1.5
            if s["d_sum"] is not None:
                d_x += s["d_sum"][b].to(d)
            d_gain += (dy * row / mean.sqrt()).sum(0)
            outs.append([d_x])
        whole = [torch.cat(parts) for parts in zip(*outs)]
        return whole + ([d_gain] if op == "norm_bwd" else [])
    if op == "quant":
        return [torch.stack([_nearest(e.to(d).view(-1, 32)).view(e.shape) for e in s["src"]])]
    if op == "dispatch":
        out = torch.zeros(s["out"].shape, dtype=d, device="cuda")
        for k in range(case["K"]):
            t = (s["slot_of"][:, k] >= 0).nonzero()[:, 0]
            e, r = s["topk_idx"][t, k].long(), s["slot_of"][t, k].long()
            out[e, r] = _nearest(s["x"][t].to(d).view(len(t), -1, 32)).view(len(t), -1)
        return [out]
    E, cap, H = s["expert_y"].shape
    I = case["I"]
    y = torch.zeros((E, cap, H), dtype=d, device="cuda")
    for e, c in enumerate(s["counts"].tolist()):
        if c:
            x = _decode(s["expert_x"], s["expert_x_scale"], e, c, False)
            h = x @ _decode(s["w_gate_up"], s["w_gate_up_scale"], e, 2 * I, True).t()
            a = _nearest((torch.nn.functional.silu(h[:, :I]) * h[:, I:]).view(c, -1, 32)).view(c, I)
            y[e, :c] = a @ _decode(s["w_down"], s["w_down_scale"], e, H, False).t()
    return [y]
