"""Cases that measure the experts' operators: the gated feed-forward over the
dispatched rows with its backward pass, the backward pass of the combine (down
to the router's logits), and the global gradient norm with clipping.

``run`` computes an operator either through this package's entry points
(``own`` true) or in its plain form: elementary torch operations in 32 bits,
rounded once at the end.  ``exact`` is the definition in 64 bits.

Notation: E experts, cap rows per expert in the padded buffers, H hidden size,
I intermediate size of an expert, N tokens with K experts each.  Expert e has
count[e] <= cap rows; rows from count[e] on are never read (they hold NaN
here) and never written (the outputs' rows stay zero).
"""
import random

import numpy as np
import torch

own = False

# Largest work of one drawn case, below the largest listed one's.
MAX_FFN_FLOPS = 2.7e12


# --- the cases ---------------------------------------------------------------

def listed():
    return [
        # One token of a Mixtral-shaped layer: two of eight experts have one row
        # each.  Batch-1 decoding: the weights of two experts are streamed once.
        dict(name="ffn_one_token", op="ffn", E=8, cap=1, H=4096, I=14336, rows=2, skew=0.0,
             draw=1, save=False),
        # Small and odd: no size is a multiple of any tile, one expert is empty,
        # gate and up are kept for a backward pass.
        dict(name="ffn_odd", op="ffn", E=5, cap=37, H=264, I=136, rows=61, skew=0.8, draw=2,
             save=True),
        # DeepSeek-V3-shaped decode step: 1024 tokens x top-8 over 256 experts,
        # about 32 rows each; bound by reading 22.5 GB of weights.
        dict(name="ffn_decode", op="ffn", E=256, cap=128, H=7168, I=2048, rows=8192, skew=0.0,
             draw=3, save=False),
        # Mixtral-shaped layer, 8 x 512 tokens, top-2: prompt or training batch,
        # bound by the tensor cores; gate and up are kept.
        dict(name="ffn_batch", op="ffn", E=8, cap=2048, H=4096, I=14336, rows=8192, skew=0.0,
             draw=4, save=True),
        # The tiny layer's backward pass: latency.
        dict(name="ffn_bwd_tiny", op="ffn_bwd", E=8, cap=64, H=256, I=256, rows=128, skew=0.0,
             draw=5, save=False),
        # Uneven experts of odd size, from none to several hundred rows.
        dict(name="ffn_bwd_uneven", op="ffn_bwd", E=32, cap=1024, H=2048, I=1000, rows=5000,
             skew=1.0, draw=6, save=False),
        # The Mixtral-shaped batch's backward pass: all three gradients.
        dict(name="ffn_bwd_batch", op="ffn_bwd", E=8, cap=2048, H=4096, I=14336, rows=8192,
             skew=0.0, draw=7, save=False),
        # Combine backward of the tiny layer: latency.
        dict(name="combine_bwd_tiny", op="combine_bwd", N=64, K=2, E=8, cap=64, H=256, masked=0.1),
        # DeepSeek-V3-shaped batch of 8192 tokens, top-8: bound by memory.
        dict(name="combine_bwd_batch", op="combine_bwd", N=8192, K=8, E=256, cap=512, H=7168,
             masked=0.0),
        # Gradients of a small layer's norms, biases and router: latency.
        dict(name="clip_small", op="clip", tensors=12, smallest=96, largest=65536, f32=0.5, draw=8,
             clips=True),
        # A whole model's worth of tensors, from a norm's gain to a projection.
        dict(name="clip_many", op="clip", tensors=300, smallest=1000, largest=4000000, f32=0.2,
             draw=9, clips=True),
        # The gradients of one Mixtral-shaped layer's experts and of its router.
        dict(name="clip_layer", op="clip", tensors=24, smallest=32768, largest=120000000, f32=0.1,
             draw=10, clips=True),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(lo * (hi / lo) ** rng.random() / step)) * step)


def draw(rng):
    op = rng.choice(["ffn", "ffn_bwd", "combine_bwd", "clip"])
    seed = rng.randrange(1 << 20)
    if op in ("ffn", "ffn_bwd"):
        while True:
            E = _log_int(rng, 1, 256)
            H = _log_int(rng, 128, 7168, 8)
            I = _log_int(rng, 128, 14336, 8)
            rows = _log_int(rng, 1, 8192)
            skew = rng.choice([0.0, 0.0, 0.5, 1.0])
            cap = min(rows, max(4, int(rows / E * (1.5 if skew == 0.0 else 4.0)) + 16))
            flops = (2 if op == "ffn" else 6) * 3.0 * rows * H * I
            padded = 6.0 * E * cap * H * I * (1 if op == "ffn" else 3)
            if flops < MAX_FFN_FLOPS and padded < 2 * MAX_FFN_FLOPS and 3 * E * H * I < 6e9:
                return dict(op=op, E=E, cap=cap, H=H, I=I, rows=rows, skew=skew, draw=seed,
                            save=op == "ffn" and rng.random() < 0.5)
    if op == "combine_bwd":
        N = _log_int(rng, 1, 8192)
        E = _log_int(rng, 2, 384)
        K = min(E, rng.choice([1, 2, 4, 6, 8]))
        H = _log_int(rng, 128, 7168, 8)
        return dict(op=op, N=N, K=K, E=E, cap=min(N, int(2.0 * N * K / E) + 24), H=H,
                    masked=rng.choice([0.0, 0.1, 0.5]))
    tensors = _log_int(rng, 1, 300)
    largest = _log_int(rng, 2000, int(min(1.0e8, 2.0e9 / tensors)))
    return dict(op=op, tensors=tensors, smallest=_log_int(rng, 1, 1000), largest=largest,
                f32=rng.choice([0.0, 0.3, 1.0]), draw=seed, clips=rng.random() < 0.7)


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


def _sizes(case):
    """Element counts of the gradient tensors and which are 32-bit."""
    rng = random.Random(case["draw"])
    lo, hi = case["smallest"], case["largest"]
    n = [max(1, int(lo * (hi / lo) ** rng.random())) for _ in range(case["tensors"])]
    n[0] = hi
    f32 = [rng.random() < case["f32"] for _ in n]
    return n, f32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, std, g, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _rows_only(t, counts, fill):
    """Fill the rows past each expert's count."""
    past = torch.arange(t.shape[1], device="cuda")[None, :] >= counts[:, None]
    t[past] = fill
    return t


def prepare(case, seed):
    g = _gen(seed)
    bf16, f32 = torch.bfloat16, torch.float32
    if case["op"] in ("ffn", "ffn_bwd"):
        E, cap, H, I = case["E"], case["cap"], case["H"], case["I"]
        counts = np.random.default_rng(int(seed)).permutation(_counts(case)).astype(np.int32)
        counts = torch.from_numpy(counts).cuda()
        nan = float("nan")
        s = dict(case=case, counts=counts,
                 expert_x=_rows_only(_normal((E, cap, H), 1.0, g), counts, nan),
                 w_gate_up=_normal((E, 2 * I, H), H ** -0.5, g),
                 w_down=_normal((E, H, I), I ** -0.5, g),
                 expert_act=torch.zeros((E, cap, I), dtype=bf16, device="cuda"))
        if case["op"] == "ffn":
            s["expert_h"] = (torch.zeros((E, cap, 2 * I), dtype=bf16, device="cuda")
                             if case["save"] else None)
            s["expert_y"] = torch.zeros((E, cap, H), dtype=bf16, device="cuda")
        else:
            # what the forward pass kept, and the gradient that arrives
            s["expert_h"] = _rows_only(_normal((E, cap, 2 * I), 1.0, g), counts, nan)
            s["d_expert_y"] = _rows_only(_normal((E, cap, H), 0.1, g), counts, nan)
            s["d_expert_h"] = torch.zeros((E, cap, 2 * I), dtype=bf16, device="cuda")
            s["d_expert_x"] = torch.zeros((E, cap, H), dtype=bf16, device="cuda")
            s["d_w_gate_up"] = torch.empty_like(s["w_gate_up"])
            s["d_w_down"] = torch.empty_like(s["w_down"])
        if own:
            import combine_moe_dispatch_gb300 as moe
            s["shape"] = moe.make_shape(1, max(1, case["rows"]), H, E, 1, cap)
            s["workspace"] = torch.zeros(moe.ffn_workspace_size(s["shape"], I), dtype=torch.uint8,
                                         device="cuda")
        return s
    if case["op"] == "combine_bwd":
        N, K, E, cap, H = case["N"], case["K"], case["E"], case["cap"], case["H"]
        idx = torch.rand((N, E), device="cuda", generator=g).argsort(1)[:, :K].contiguous()
        drop = torch.rand((N, K), device="cuda", generator=g) < case["masked"]
        idx[drop] = -1
        flat = idx.reshape(-1)
        order = torch.argsort(flat, stable=True)
        first = torch.searchsorted(flat[order].contiguous(), flat)
        slot = torch.empty_like(flat)
        slot[order] = torch.arange(N * K, device="cuda")
        slot = slot - first
        out = (flat < 0) | (slot >= cap)          # not routed, or dropped at capacity
        slot[out] = -1
        flat = torch.where(out, torch.full_like(flat, -1), flat)
        s = dict(case=case, topk_idx=flat.reshape(N, K).int(), slot_of=slot.reshape(N, K).int(),
                 topk_weights=torch.softmax(_normal((N, K), 1.0, g, f32), 1),
                 d_y=_normal((N, H), 0.1, g), expert_y=_normal((E, cap, H), 1.0, g),
                 d_expert_y=torch.zeros((E, cap, H), dtype=bf16, device="cuda"),
                 d_weights=torch.empty((N, K), dtype=f32, device="cuda"),
                 d_logits=torch.empty((N, E), dtype=f32, device="cuda"))
        if own:
            import combine_moe_dispatch_gb300 as moe
            s["shape"] = moe.make_shape(1, N, H, E, K, cap)
            s["workspace"] = torch.zeros(moe.workspace_size(s["shape"]), dtype=torch.uint8,
                                         device="cuda")
        return s
    n, is32 = _sizes(case)
    dtypes = [f32 if a else bf16 for a in is32]
    grads = [_normal((m,), 0.01, g, dt) for m, dt in zip(n, dtypes)]
    # the clipped gradients, side by side in one buffer of each type
    place, used = [], {f32: 0, bf16: 0}
    for m, dt in zip(n, dtypes):
        place.append(used[dt])
        used[dt] += (m + 15) // 16 * 16
    flat = {dt: torch.zeros(used[dt], dtype=dt, device="cuda") for dt in (f32, bf16)}
    s = dict(case=case, grads=grads, max_norm=1.0 if case["clips"] else 1e6,
             outs=[flat[dt][p:p + m] for m, dt, p in zip(n, dtypes, place)],
             flat=[flat[dt] for dt in (f32, bf16) if used[dt]],
             norm=torch.zeros((), dtype=f32, device="cuda"))
    if own:
        import combine_moe_dispatch_gb300 as moe
        s["workspace"] = torch.zeros(moe.clip_workspace_size(), dtype=torch.uint8, device="cuda")
    return s


# --- one pass ----------------------------------------------------------------

def _run_own(s):
    import combine_moe_dispatch_gb300 as moe
    op = s["case"]["op"]
    if op == "ffn":
        moe.ffn(s["shape"], s["case"]["I"], s["expert_x"], s["w_gate_up"], s["w_down"], s["counts"],
                s["expert_h"], s["expert_act"], s["expert_y"], s["workspace"])
        return [s["expert_y"]] + ([s["expert_h"]] if s["case"]["save"] else [])
    if op == "ffn_bwd":
        moe.ffn_backward(s["shape"], s["case"]["I"], s["d_expert_y"], s["expert_x"], s["expert_h"],
                         s["w_gate_up"], s["w_down"], s["counts"], s["expert_act"], s["d_expert_h"],
                         s["d_expert_x"], s["d_w_gate_up"], s["d_w_down"], s["workspace"])
        return [s["d_expert_x"], s["d_w_gate_up"], s["d_w_down"]]
    if op == "combine_bwd":
        moe.combine_backward(s["shape"], s["d_y"], s["expert_y"], s["topk_idx"], s["slot_of"],
                             s["topk_weights"], s["d_expert_y"], s["d_weights"], s["d_logits"],
                             s["workspace"])
        return [s["d_expert_y"], s["d_weights"], s["d_logits"]]
    moe.clip_grad_norm(s["grads"], s["outs"], s["max_norm"], s["norm"], s["workspace"])
    return [s["norm"]] + s["flat"]


def _below(t, counts):
    """[E, cap, 1]: which rows exist."""
    return (torch.arange(t.shape[1], device=t.device)[None, :] < counts[:, None])[:, :, None]


def _existing(t, counts):
    return torch.where(_below(t, counts), t, torch.zeros((), dtype=t.dtype, device=t.device)).float()


def _plain_ffn(s):
    I, bf16 = s["case"]["I"], torch.bfloat16
    x = _existing(s["expert_x"], s["counts"])
    h = torch.bmm(x, s["w_gate_up"].float().transpose(1, 2))
    gate, up = h[:, :, :I], h[:, :, I:]
    a = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.bmm(a, s["w_down"].float().transpose(1, 2)).to(bf16)
    return [y] + ([h.to(bf16)] if s["case"]["save"] else [])


def _plain_ffn_bwd(s):
    I, bf16 = s["case"]["I"], torch.bfloat16
    dy = _existing(s["d_expert_y"], s["counts"])
    h = _existing(s["expert_h"], s["counts"])
    gate, up = h[:, :, :I], h[:, :, I:]
    sig = 1.0 / (1.0 + torch.exp(-gate))
    silu = gate * sig
    d_w_down = torch.bmm(dy.transpose(1, 2), silu * up).to(bf16)
    da = torch.bmm(dy, s["w_down"].float())
    dh = torch.cat([da * up * sig * (1.0 + gate * (1.0 - sig)), da * silu], 2)
    d_w_gate_up = torch.bmm(dh.transpose(1, 2), _existing(s["expert_x"], s["counts"])).to(bf16)
    d_x = torch.bmm(dh, s["w_gate_up"].float()).to(bf16)
    return [d_x, d_w_gate_up, d_w_down]


def _plain_combine_bwd(s):
    E, cap, H = s["expert_y"].shape
    N, K = s["topk_idx"].shape
    routed = s["slot_of"] >= 0
    row = torch.where(routed, s["topk_idx"] * cap + s["slot_of"], 0).long()
    dy = s["d_y"].float()
    w = torch.where(routed, s["topk_weights"], 0.0)
    dw = (s["expert_y"].view(E * cap, H)[row].float() * dy[:, None, :]).sum(2)
    dw = torch.where(routed, dw, 0.0)
    at = row[routed]
    d_rows = (w[:, :, None] * dy[:, None, :]).to(torch.bfloat16)[routed]
    d_expert_y = torch.zeros((E * cap, H), dtype=torch.bfloat16, device="cuda")
    d_expert_y[at] = d_rows
    dl = w * (dw - (w * dw).sum(1, keepdim=True))
    d_logits = torch.zeros((N, E), device="cuda")
    d_logits.scatter_add_(1, torch.where(routed, s["topk_idx"], 0).long(), dl)
    return [d_expert_y.view(E, cap, H), dw, d_logits]


def _plain_clip(s):
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    [o.copy_(t.float() * coef) for o, t in zip(s["outs"], s["grads"])]
    return [norm] + s["flat"]


PLAIN = {"ffn": _plain_ffn, "ffn_bwd": _plain_ffn_bwd, "combine_bwd": _plain_combine_bwd,
         "clip": _plain_clip}


def run(s):
    return _run_own(s) if own else PLAIN[s["case"]["op"]](s)


# --- what a pass cannot do without --------------------------------------------

def work(case):
    if case["op"] in ("ffn", "ffn_bwd"):
        counts = _counts(case)
        rows, active = int(counts.sum()), int((counts > 0).sum())
        E, H, I = case["E"], case["H"], case["I"]
        weights = 3 * H * I * 2
        if case["op"] == "ffn":
            kept = 4 * I * rows if case["save"] else 0
            return {"bytes": active * weights + 4 * H * rows + kept, "flops": 6.0 * rows * H * I}
        return {"bytes": active * weights + E * weights + (6 * H + 4 * I) * rows,
                "flops": 12.0 * rows * H * I}
    if case["op"] == "combine_bwd":
        N, K, E, H = case["N"], case["K"], case["E"], case["H"]
        routed = N * K * (1.0 - case["masked"])
        return {"bytes": 2 * N * H + 4 * routed * H + 16 * N * K + 4 * N * E,
                "flops": 3.0 * routed * H}
    n, is32 = _sizes(case)
    data = sum(m * (4 if a else 2) for m, a in zip(n, is32))
    return {"bytes": 2 * data, "flops": 3.0 * sum(n)}


# --- the definition in 64 bits -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] in ("ffn", "ffn_bwd"):
        E, cap, H, I = case["E"], case["cap"], case["H"], case["I"]
        counts = s["counts"].tolist()
        if case["op"] == "ffn":
            y = torch.zeros((E, cap, H), dtype=d, device="cuda")
            h_out = torch.zeros((E, cap, 2 * I), dtype=d, device="cuda") if case["save"] else None
            for e, c in enumerate(counts):
                if c:
                    h = s["expert_x"][e, :c].to(d) @ s["w_gate_up"][e].to(d).t()
                    y[e, :c] = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ s["w_down"][e].to(d).t()
                    if case["save"]:
                        h_out[e, :c] = h
            return [y] + ([h_out] if case["save"] else [])
        d_x = torch.zeros((E, cap, H), dtype=d, device="cuda")
        d_up = torch.zeros((E, 2 * I, H), dtype=d, device="cuda")
        d_down = torch.zeros((E, H, I), dtype=d, device="cuda")
        for e, c in enumerate(counts):
            if c:
                g = s["expert_h"][e, :c, :I].to(d)
                u = s["expert_h"][e, :c, I:].to(d)
                dy = s["d_expert_y"][e, :c].to(d)
                sig = torch.sigmoid(g)
                da = dy @ s["w_down"][e].to(d)
                dh = torch.cat([da * u * (sig + g * sig * torch.sigmoid(-g)), da * g * sig], 1)
                d_down[e] = dy.t() @ (g * sig * u)
                d_up[e] = dh.t() @ s["expert_x"][e, :c].to(d)
                d_x[e, :c] = dh @ s["w_gate_up"][e].to(d)
        return [d_x, d_up, d_down]
    if case["op"] == "combine_bwd":
        N, K, E, H = case["N"], case["K"], case["E"], case["H"]
        de = torch.zeros(s["expert_y"].shape, dtype=d, device="cuda")
        dw = torch.zeros((N, K), dtype=d, device="cuda")
        dl = torch.zeros((N, E), dtype=d, device="cuda")
        w = s["topk_weights"].to(d)
        tokens = torch.arange(N, device="cuda")
        for k in range(K):
            t = tokens[s["slot_of"][:, k] >= 0]
            e, r = s["topk_idx"][t, k].long(), s["slot_of"][t, k].long()
            for a in range(0, len(t), 1024):
                b = slice(a, a + 1024)
                dy = s["d_y"][t[b]].to(d)
                dw[t[b], k] = (dy * s["expert_y"][e[b], r[b]].to(d)).sum(1)
                de[e[b], r[b]] = w[t[b], k, None] * dy
        on = (s["slot_of"] >= 0).to(d)
        mean = (on * w * dw).sum(1)
        for k in range(K):
            t = tokens[s["slot_of"][:, k] >= 0]
            dl[t, s["topk_idx"][t, k].long()] = w[t, k] * (dw[t, k] - mean[t])
        return [de, dw, dl]
    total = sum(float(t.to(d).square().sum()) for t in s["grads"])
    norm = total ** 0.5
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    flats = []
    for dt in (torch.float32, torch.bfloat16):
        parts = []
        for t in s["grads"]:
            if t.dtype == dt:
                pad = -t.numel() % 16
                parts.append(torch.nn.functional.pad(t.to(d) * coef, (0, pad)))
        if parts:
            flats.append(torch.cat(parts))
    return [torch.tensor(norm, dtype=d, device="cuda")] + flats
